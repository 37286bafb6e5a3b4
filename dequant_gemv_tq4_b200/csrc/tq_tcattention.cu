// tq_tcattention.cu -- attention over the TQ4_1S cache for many rows (drafted
// trees) on the fifth-generation tensor cores.  Mathematics and the split of
// the work: tq_attention.cu; here a group is a tile of 128 tokens, a worker a CTA.
//
// One CTA per SM holds two streams of work, each with 128 query rows in shared
// memory, a 128 x 128 score accumulator and an output accumulator in tensor
// memory.  With more than 128 rows the streams are two row tiles over the same
// tokens (records are decoded once for 256 rows); with fewer they take even
// and odd token tiles of one row tile and leave two partial results.
//   decode warps   codes to fp16 centroid x scale into the 128-byte-swizzled
//                  operand layout, two stages of 128 tokens for keys and for
//                  values; seven warps take pieces of 32 tokens in turn
//   one warp       issues S = Q K^T (both operands in shared memory, K-major)
//                  and O += P V (P from tensor memory, V as it was written,
//                  tokens as rows: the instruction takes it N-major)
//   softmax warps  one thread per row: scores from tensor memory, running
//                  maximum (followed lazily) and sum, weights as fp16 back into
//                  the score's own columns
// While one stream's softmax runs, the tensor cores work for the other.
//
// What bounds it: the chain scores - softmax - weights - product of the two
// streams, with the exponentials (one per row and token, 40% of their unit's
// peak), the decoding (ALU pipe 38%) and the tensor pipe (40%) all less than
// half used.  4 sequences of 16384 tokens, 64 drafted tokens, 64 query over 8
// key/value heads of 128: 157.5 us with the joining launch, 875 TFLOP/s, at the
// full clock of a burst (1965 MHz); 174 us once a second of such calls has brought
// the GPU to its power limit (992 W, 1770 MHz).  16 sequences of up to 4000 tokens
// with 64 rows a head 51.5 us: a CTA's share is about sixteen tiles in one or two
// parts, and a part's beginning and end (last product, results out, next query
// rotated, first score), which nothing overlaps, counts as four tiles; half of
// each 128-row product is padding there.
// Forms measured when this one took 171 us for the large case: 64-token tiles
// with two score buffers a stream 201; weights handed over in halves 188; a
// second issuing warp 207.  Seven decode warps, the eighth warp of their register
// share issues; eight in a CTA of 20 warps took 178.
#include "tq_attention.cuh"

namespace tq {

namespace {

constexpr int kTile = 128;      // tokens of a tile
constexpr int kRowTile = 128;   // rows of a stream
constexpr int kSoftWarps = 8;   // warps 0..7: four per stream
constexpr int kDecodeWarps = 7; // warps 8..11 and 13..15
constexpr int kMmaWarp = 12;    // issue
constexpr int kTcaThreads = 512;
constexpr int kPieces = 8;      // of a tile: 32 tokens' keys or values
// Registers a thread: 128 at launch; the softmax holds a whole row of scores.
// Shares of the launch's 65536: 256 * 184 + 256 * 72 = 65536.
constexpr int kSoftRegs = 184, kOtherRegs = 72;
static_assert(256 * kSoftRegs + 256 * kOtherRegs <= kTcaThreads * 128, "register shares");
// setmaxnreg has to be the same instruction for all four warps of a warpgroup:
// the shares change hands where whole warpgroups part, above the roles.
static_assert(kSoftWarps % 4 == 0 && kTcaThreads / 32 % 4 == 0, "shares go by warpgroups");
constexpr int kTmemCols = 512;
constexpr uint32_t kOCol = 256;  // output accumulators; scores at 0 and 128
constexpr unsigned kStatusTimeout = 1u;
constexpr unsigned kStatusTmem = 4u;

// Byte offsets from the 1024-aligned start of dynamic shared memory.
template <int D>
struct TcaShape {
    static constexpr uint32_t kHalf = 128 * 128;        // 128 rows of 64 fp16
    static constexpr uint32_t kOperand = kHalf * (D / 64);
    static constexpr uint32_t kQ = 0;                   // two row tiles
    static constexpr uint32_t kK = kQ + 2 * kOperand;   // two stages
    static constexpr uint32_t kV = kK + 2 * kOperand;   // two stages
    static constexpr uint32_t kBars = kV + 2 * kOperand;
    static constexpr uint32_t kTmemSlot = kBars + 8 * 16;
    static constexpr uint32_t kStatus = kTmemSlot + 8;
    static constexpr uint32_t kScan = kTmemSlot + 16;
    static constexpr uint32_t kPrefix = kScan + 32 * 4;
    static constexpr uint32_t kEnd = kPrefix + (kAttnMaxBatch + 1) * 4;
    static constexpr int kBytes = (int)kEnd + 1024;     // room for the alignment
    static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
    // fp32 accumulator, fp16 operands, M = 128; bit 16: B is N-major
    static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
    static constexpr uint32_t kIdescO =
        (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
};

// barriers
enum : int { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPReady = 10, kODone = 12, kLast = 13 };

// ---- PTX wrappers ------------------------------------------------------------
template <int N>
__device__ __forceinline__ void a_regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void a_regs_fewer() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void a_mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool a_mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Wait for phase `parity`; false after `limit` cycles (or 2^30 polls).  The
// limit is read from the SM's own clock and only now and then: reading the
// global timer between polls delayed every wait of the pipeline.
__device__ __forceinline__ bool a_mbar_wait(uint32_t bar, uint32_t parity, long long limit) {
    if (a_mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        if (a_mbar_try(bar, parity)) return true;
        if ((it & 63u) == 63u && clock64() - t0 > limit) return false;
    }
    return false;
}
__device__ __forceinline__ bool a_mbar_wait_warp(uint32_t bar, uint32_t parity, long long limit) {
    return __all_sync(kFull, a_mbar_wait(bar, parity, limit));
}
__device__ __forceinline__ void a_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void a_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void a_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void a_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void a_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void a_sts128(uint32_t a, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ uint4 a_lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// One lane of the (whole) warp, the same one every time.
__device__ __forceinline__ bool a_elect() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void a_named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// D (tensor memory) [+]= A (shared memory) x B (shared memory)
__device__ __forceinline__ void a_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D (tensor memory) [+]= A (tensor memory) x B (shared memory)
__device__ __forceinline__ void a_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 consecutive 32-bit columns of this thread's tensor-memory lane; the
// registers are defined after the next a_wait_ld.
__device__ __forceinline__ void a_ld32(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void a_ld16(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void a_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void a_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void a_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Operand descriptor, 128-byte swizzle, version 1.  K-major: 8-row groups
// 1024 bytes apart (lbo unused).  N-major: 64-element groups along N `lbo`
// apart, 8-row (k) groups 1024 bytes apart.
__device__ __forceinline__ uint64_t a_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Address of 16-byte chunk `chunk` (0..7) of row r in a 128-byte-swizzled half.
__device__ __forceinline__ uint32_t swizzled(uint32_t half, int r, int chunk) {
    return half + (uint32_t)r * 128u + (uint32_t)((chunk ^ (r & 7)) << 4);
}

// A worker's part of a unit: tiles [ta, tb) of a (sequence, head, row tile).
struct Part {
    int b, head, row0, len, n, ta, tb;
    bool last;  // the unit ends with it
    int64_t unit;
};

template <int D>
struct Walk {  // the parts of a worker's range, the same for every warp
    const int *prefix;
    int per_seq;
    int64_t at, end;
    __device__ __forceinline__ bool next(const AttnParams &P, Part &p) {
        while (at < end) {
            int lo = 0, hi = P.c.batch - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((int64_t)prefix[mid] * per_seq <= at) lo = mid;
                else hi = mid - 1;
            }
            const int groups = prefix[lo + 1] - prefix[lo];
            const int64_t in_seq = at - (int64_t)prefix[lo] * per_seq;
            const int hr = (int)quotient(in_seq, groups);
            const int va = (int)(in_seq - (int64_t)hr * groups);
            const int vb = (int)min((int64_t)groups, va + (end - at));
            at += vb - va;
            p.ta = max(va - P.extra, 0);
            p.tb = max(vb - P.extra, 0);
            if (p.ta >= p.tb) continue;
            p.last = vb == groups;
            p.b = lo;
            p.head = hr / P.row_tiles;
            p.row0 = hr % P.row_tiles * P.tile_rows;
            p.unit = (int64_t)lo * per_seq + hr;
            const int len = P.lens[lo];
            p.n = seq_tokens(P, len);
            p.len = min(max(len, 0), P.c.pages_per_seq << P.c.page_shift);
            return true;
        }
        return false;
    }
};

// ---- decode: codes of one token's D / 2 elements to swizzled fp16 ------------
// A lane owns one token of a piece: D / 32 blocks of 32 elements.
template <int D>
struct TokenRegs {
    uint4 w[D / 32];
    uint32_t d[D / 32];
};

template <int D>
__device__ __forceinline__ void load_token(const AttnParams &P, int64_t rec, bool valid, TokenRegs<D> &r) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        r.w[i] = make_uint4(0u, 0u, 0u, 0u);
        r.d[i] = 0;
    }
    if (valid) {
        const uint4 *codes = reinterpret_cast<const uint4 *>(P.c.codes + rec * (D / 2));
        const uint2 *scales = reinterpret_cast<const uint2 *>(P.c.scales + rec * (D / 16));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) r.w[i] = ld(codes + i);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const uint2 d = ld(scales + i);
            r.d[2 * i] = d.x;
            r.d[2 * i + 1] = d.y;
        }
    }
}

template <int D>
__device__ __forceinline__ void decode_token(const TokenRegs<D> &r, uint32_t operand, int row) {
#pragma unroll
    for (int blk = 0; blk < D / 32; ++blk) {
        const uint32_t half = operand + (uint32_t)(blk >> 1) * TcaShape<D>::kHalf;
        const uint32_t w[4] = {r.w[blk].x, r.w[blk].y, r.w[blk].z, r.w[blk].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // eight elements, 16 bytes
            const uint32_t d2 = prmt(r.d[blk], r.d[blk], j < 2 ? 0x1010u : 0x3232u);
            uint32_t o[4];
            decode_word(w[j], o);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = hmul2(o[k], d2);
            a_sts128(swizzled(half, row, (blk & 1) * 4 + j), o);
        }
    }
}

// ---- query rows: rotated, fp16, swizzled ---------------------------------------
// Blocks [b0, b1) of a row; returns the unit of its scores.  All of the row is
// asked for at once, because its largest element has to be known first; a row of
// 16-bit elements waits in its place in the operand (as long as what replaces
// it), one of fp32 is read again.  The blocks come one at a time: what runs once
// per part costs the fetch of its code more than its arithmetic.
template <int DT, int D>
__device__ __forceinline__ float rotate_row(const AttnParams &P, int64_t x, bool valid, uint32_t operand, int row,
                                            int b0, int b1) {
    constexpr int E = ElemSize<DT>::value, C = D * E / 16;  // 16-byte chunks of the row
    const uint4 *at = reinterpret_cast<const uint4 *>(P.q + x * E);
    auto place = [&](int blk, int j) {  // of chunk j of a block
        return swizzled(operand + (uint32_t)(blk >> 1) * TcaShape<D>::kHalf, row, (blk & 1) * 4 + j);
    };
    float most = 0.f;
    {
        uint4 raw[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (valid) raw[i] = ld(at + i);
        }
        uint32_t most2 = 0;  // of 16-bit elements: magnitudes are ordered as whole numbers
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (DT == kF32) most = fmaxf(most, fabsf(__uint_as_float(w[k])));
                else most2 = __vmaxu2(most2, w[k] & 0x7FFF7FFFu);
            }
            if (DT != kF32 && i / 4 >= b0 && i / 4 < b1) a_sts128(place(i / 4, i % 4), w);
        }
        if (DT != kF32) {
            most2 = max(most2 >> 16, most2 & 0xFFFFu);
            most = DT == kBF16 ? __uint_as_float(most2 << 16) : __half2float(__ushort_as_half((unsigned short)most2));
        }
    }
    const RowScale scale(P.q_factor, most);
#pragma unroll 1
    for (int blk = b0; blk < b1; ++blk) {
        const uint32_t bits = c_sign_words.w[blk];
        float v[32];
        if (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (valid) q = ld(at + 8 * blk + i);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 * i + k] = __uint_as_float(w[k]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 q = a_lds128(place(blk, j));
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (DT == kBF16) {
                        v[8 * j + 2 * k] = __uint_as_float(w[k] << 16);
                        v[8 * j + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                        v[8 * j + 2 * k] = f.x;
                        v[8 * j + 2 * k + 1] = f.y;
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = flip(v[e], (bits << (31 - e)) & 0x80000000u);
#pragma unroll
        for (int h = 1; h < 32; h <<= 1)
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if ((e & h) == 0) {
                    const float a = v[e], b = v[e + h];
                    v[e] = a + b;
                    v[e + h] = a - b;
                }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2 h =
                    __floats2half2_rn(v[8 * j + 2 * k] * scale.factor, v[8 * j + 2 * k + 1] * scale.factor);
                o[k] = *reinterpret_cast<const uint32_t *>(&h);
            }
            a_sts128(place(blk, j), o);
        }
    }
    return scale.unit;
}

// ---- softmax of one row's 128 scores ---------------------------------------------
// Packed fp32 pairs: each half one IEEE operation.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// Output sums of this thread's row times f.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t t_o, float f) {
#pragma unroll 1
    for (int k = 0; k < D; k += 16) {  // (a whole row of scores is in registers meanwhile)
        uint32_t v[16];
        a_ld16(t_o + (uint32_t)k, v);
        a_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
        a_st16(t_o + (uint32_t)k, v);
    }
}

// The maximum of 128 scores.
__device__ __forceinline__ float max128(const uint32_t *v) {
    float x[4] = {kNoMax, kNoMax, kNoMax, kNoMax};
#pragma unroll
    for (int e = 0; e < 128; e += 2)
        x[(e >> 1) & 3] = fmaxf(x[(e >> 1) & 3], fmaxf(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
}

// Weights of 128 scores into 64 columns at t_p, their sum onto `sum`.
__device__ __forceinline__ void weights128(uint32_t *v, uint64_t unit2, uint64_t off2, uint32_t t_p,
                                           uint64_t (&sum)[2]) {
#pragma unroll
    for (int e = 0; e < 128; e += 2) {
        float a, b;
        unpack2(fma2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), unit2, off2), a, b);
        a = ex2(a);
        b = ex2(b);
        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pack2(a, b));
        const __half2 h = __floats2half2_rn(a, b);
        v[e / 2] = *reinterpret_cast<const uint32_t *>(&h);
        if ((e & 31) == 30) a_st16(t_p + (e >> 5) * 16u, v + (e >> 5) * 16);
    }
}

// `off` follows to a maximum mx of the scores where one of the warp's rows has
// outgrown it.  `have`: the output sums hold earlier products.
template <int D>
__device__ __forceinline__ void follow(uint32_t t_o, float unit, bool have, float mx, float &off, float &l) {
    if (__any_sync(kFull, outgrown(mx, unit, off))) {
        const float lower = fminf(off, weight_offset(mx, unit));
        const float f = ex2(lower - off);
        off = lower;
        l *= f;
        // the scores' commit followed this stream's last product: its sums are complete
        if (have) rescale_row<D>(t_o, f);
    }
}

__device__ __forceinline__ float sum_of(const uint64_t (&sum)[2]) {
    float s0, s1, s2, s3;
    unpack2(sum[0], s0, s1);
    unpack2(sum[1], s2, s3);
    return (s0 + s1) + (s2 + s3);
}

// Scores at t_s to weights in the first half of their columns; the whole row is
// in registers between.
template <int D>
__device__ __forceinline__ void softmax_row(uint32_t t_s, uint32_t t_o, float unit, bool have, float &off, float &l) {
    uint32_t v[128];
#pragma unroll
    for (int k = 0; k < 4; ++k) a_ld32(t_s + 32u * k, v + 32 * k);
    a_wait_ld();
    follow<D>(t_o, unit, have, max128(v), off, l);
    const uint64_t unit2 = pack2(unit, unit), off2 = pack2(off, off);
    uint64_t sum[2] = {0, 0};
    weights128(v, unit2, off2, t_s, sum);
    l += sum_of(sum);
    a_wait_st();
}

// Which of a tile's columns a row sees: the context's `full` columns, then
// drafted token j where bit j of `see` is set; bit g of `groups`: columns
// 16 g .. have a page.  Word k: columns 32 k ...
__device__ __forceinline__ uint32_t column_word(int k, int full, uint64_t see, uint32_t groups) {
    const int f = full - 32 * k;  // the context's columns from this word's start
    uint32_t w;
    if (f >= 32) w = ~0u;
    else if (f > 0) w = ((uint32_t)see << f) | ((1u << f) - 1u);
    else w = f > -64 ? (uint32_t)(see >> -f) : 0u;
    const uint32_t g = groups >> (2 * k);
    return w & ((g & 1u ? 0xFFFFu : 0u) | (g & 2u ? 0xFFFF0000u : 0u));
}

// The same for a tile with columns that do not count (a sequence's last one or
// two tiles), 32 columns at a time.
template <int D>
__device__ __forceinline__ void softmax_row_masked(uint32_t t_s, uint32_t t_o, float unit, bool have, int full,
                                                   uint64_t see, uint32_t groups, float &off, float &l) {
    float mx = kNoMax;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        uint32_t v[32];
        a_ld32(t_s + 32u * k, v);
        const uint32_t w = column_word(k, full, see, groups);
        a_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) mx = (w >> e) & 1u ? fmaxf(mx, __uint_as_float(v[e])) : mx;
    }
    follow<D>(t_o, unit, have, mx, off, l);
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        uint32_t v[32];
        a_ld32(t_s + 32u * k, v);
        const uint32_t w = column_word(k, full, see, groups);
        a_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float a = ex2(fmaf(__uint_as_float(v[e]), unit, off));
            float b = ex2(fmaf(__uint_as_float(v[e + 1]), unit, off));
            if (!((w >> e) & 1u)) a = 0.f;
            if (!((w >> (e + 1)) & 1u)) b = 0.f;
            l += a + b;
            const __half2 h = __floats2half2_rn(a, b);
            v[e / 2] = *reinterpret_cast<const uint32_t *>(&h);
        }
        a_st16(t_s + 16u * k, v);  // over scores that are read by now
    }
    a_wait_st();
}

template <int D>
__global__ void __launch_bounds__(kTcaThreads, 1) tc_attend_kernel(const AttnParams P) {
    using S = TcaShape<D>;
    extern __shared__ char smem_raw[];
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    char *smem = smem_raw + (base - raw);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);
    int *prefix = reinterpret_cast<int *>(smem + S::kPrefix);
    auto bar = [&](int i) { return base + S::kBars + 8u * (uint32_t)i; };
    // this CTA's status, for the joining launch: a word in the header would have
    // to be cleared before any CTA reports, and nothing orders the CTAs
    unsigned *status = reinterpret_cast<unsigned *>(smem + S::kStatus);
    if (tid == 0) {
        *status = 0u;
        for (int i = 0; i < 2; ++i) {
            a_mbar_init(bar(kKFull + i), kPieces / 2);
            a_mbar_init(bar(kKEmpty + i), 1);
            a_mbar_init(bar(kVFull + i), kPieces / 2);
            a_mbar_init(bar(kVEmpty + i), 1);
            a_mbar_init(bar(kSFull + i), 1);
            a_mbar_init(bar(kPReady + i), kSoftWarps / 2);
        }
        a_mbar_init(bar(kODone), 1);
        a_mbar_init(bar(kLast), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + S::kTmemSlot),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    grid_dependents_launch();  // the joining launch; it waits for this one's end
    a_fence_before();
    scan_sequences(P, prefix, reinterpret_cast<int *>(smem + S::kScan), tid, kTcaThreads);
    a_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + S::kTmemSlot);
    // all 512 columns: the base is lane 0, column 0 (checked, never expected)
    const bool tmem_ok = tmem == 0u && !(P.inject_tmem && blockIdx.x == gridDim.x - 1);
    if (!tmem_ok && tid == 0) atomicOr(status, kStatusTmem);

    Walk<D> walk;
    walk.prefix = prefix;
    walk.per_seq = P.c.kv_heads * P.row_tiles;
    const int64_t W = (int64_t)prefix[P.c.batch] * walk.per_seq;
    const int workers = worker_count(P, W);
    const int me = blockIdx.x;
    walk.at = me < workers ? quotient(W * me, workers) : 0;
    walk.end = me < workers ? quotient(W * (me + 1), workers) : 0;
    const bool pair = P.tile_rows == 2 * kRowTile;  // the streams are two row tiles
    bool ok = tmem_ok;
    auto give_up = [&]() {
        ok = false;
        atomicOr(status, kStatusTimeout);
    };
    Part p;

    if (warp < kSoftWarps) a_regs_more<kSoftRegs>();
    else a_regs_fewer<kOtherRegs>();

    if (warp < kSoftWarps) {
        // ---- softmax: thread = row of a stream ----------------------------------
        const int s = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + 128u * s, t_o = tmem + lanes + kOCol + 128u * s;
        uint32_t jobs_done = 0, parts_done = 0;
        const int shift = P.c.page_shift;
        while (walk.next(P, p)) {
            float unit;  // of this row's scores
            // the query rows: this stream's tile, or half of the common one's blocks
            {
                const int q_row = p.row0 + (pair ? s * kRowTile : 0) + row;
                const bool valid = q_row < P.rows;
                const int t = valid ? q_row / P.group_heads : 0;
                const int h = p.head * P.group_heads + (valid ? q_row % P.group_heads : 0);
                const int64_t x = p.b * P.q_batch + t * P.q_token + h * P.q_head;
                const uint32_t operand = base + S::kQ + (pair ? s : 0) * S::kOperand;
                constexpr int kBlocks = D / 32;
                const int b0 = pair ? 0 : s * (kBlocks / 2), b1 = pair ? kBlocks : b0 + kBlocks / 2;
                if (P.qdtype == kF32) unit = rotate_row<kF32, D>(P, x, valid, operand, row, b0, b1);
                else if (P.qdtype == kBF16) unit = rotate_row<kBF16, D>(P, x, valid, operand, row, b0, b1);
                else unit = rotate_row<kF16, D>(P, x, valid, operand, row, b0, b1);
                a_proxy_fence();
            }
            a_named_sync(1, (kSoftWarps + 1) * 32);

            const int out_row = pair ? s * kRowTile + row : row;  // of the partial result
            const int unit_row = p.row0 + out_row;
            const bool any_rows = unit_row - lane < P.rows;
            const TreeWords words(P, TreeParents(P, p.b, lane), lane);
            const uint64_t see = words.of(min(unit_row / P.group_heads, P.tree - 1));
            const int32_t *table = P.c.page_table + p.b * P.c.table_ld;
            const int tiles = p.tb - p.ta, jobs = pair ? 2 * tiles : tiles;
            float off = weight_offset(kNoMax, unit), l = 0.f;
            int seen_jobs = 0;
            for (int i = s; i < jobs && ok; i += 2, ++seen_jobs) {
                const int tile = p.ta + (pair ? i >> 1 : i);
                // which groups of 16 tokens have a page
                int page = -1;
                const int place = tile * kTile + (lane & 7) * 16;
                if (place < p.n) page = table[place >> shift];
                const uint32_t groups = __ballot_sync(kFull, page >= 0 && page < P.c.pages) & 0xFFu;
                const bool tail = tile * kTile + kTile > p.len || groups != 0xFFu;
                if (!a_mbar_wait_warp(bar(kSFull + s), jobs_done & 1u, P.timeout_cycles)) {
                    give_up();
                    break;
                }
                a_fence_after();
                if (!any_rows) {
                    // no row of this warp is asked for: whatever stands in its lanes stays there
                } else if (tail)
                    softmax_row_masked<D>(t_s, t_o, unit, seen_jobs > 0, p.len - tile * kTile, see, groups, off, l);
                else
                    softmax_row<D>(t_s, t_o, unit, seen_jobs > 0, off, l);
                a_fence_before();
                __syncwarp();
                if (lane == 0) a_arrive(bar(kPReady + s));
                ++jobs_done;
            }
            // the part's result
            if (ok && !a_mbar_wait_warp(bar(kODone), parts_done & 1u, P.timeout_cycles)) give_up();
            ++parts_done;
            if (ok) {
                a_fence_after();
                if (tid == 0 && p.ta == 0) P.span[2 * p.unit] = me;
                if (tid == 0 && p.last) P.span[2 * p.unit + 1] = me;
                const int64_t slot = (p.unit + me) * P.parts + (pair ? 0 : s);
                const int64_t row0 = slot * P.tile_rows + out_row - lane;  // of this warp
                // a token that is not there answers zero
                if (unit_row < P.rows)
                    reinterpret_cast<float2 *>(P.part_ml)[row0 + lane] = make_float2(-off, see == 0 ? 0.f : l);
                // rows leave through this warp's quarter of its stream's query
                // tile (every product has read it), 32 elements of 32 rows at a
                // time, so that a store covers whole 128-byte lines of four rows
                const uint32_t stage = base + S::kQ + (uint32_t)s * S::kOperand + (uint32_t)(warp & 3) * 4096u;
                const int rows = min(32, P.rows - (unit_row - lane));
#pragma unroll 1
                for (int k = 0; k < D && seen_jobs > 0 && any_rows; k += 32) {
                    uint32_t v[32];
                    a_ld32(t_o + (uint32_t)k, v);
                    a_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t w[4] = {v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]};
                        a_sts128(swizzled(stage, lane, j), w);
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = 4 * j + (lane >> 3);
                        if (r < rows)
                            *reinterpret_cast<uint4 *>(P.part_o + (row0 + r) * D + k + 4 * (lane & 7)) =
                                a_lds128(swizzled(stage, r, lane & 7));
                    }
                    __syncwarp();
                }
                a_fence_before();
            }
            a_named_sync(1, (kSoftWarps + 1) * 32);  // the queries may be replaced
        }
    } else if (warp != kMmaWarp) {
        // ---- decode ------------------------------------------------------------------
        const int first = warp < kMmaWarp ? warp - kSoftWarps : warp - kSoftWarps - 1;  // of this warp's pieces
        const int shift = P.c.page_shift, in_page = (1 << shift) - 1;
        const int v_rows = P.c.kv_heads << shift;
        uint32_t tile_no = 0, piece = (uint32_t)first;  // of the walk
        while (ok && walk.next(P, p)) {
            const int32_t *table = P.c.page_table + p.b * P.c.table_ld;
            const uint32_t end = (tile_no + (uint32_t)(p.tb - p.ta)) * kPieces;
            uint64_t present = 0;
            bool known = false;
            // piece i: tile i / 8 of the walk, its keys or values, 32 rows
            auto place_of = [&](uint32_t i) {
                return (p.ta + (int)(i / kPieces - tile_no)) * kTile + (int)(i & 3u) * 32 + lane;
            };
            // Page of this lane's token; none for a record that no row sees, which
            // then counts as zero whatever the memory holds.
            auto page_of = [&](uint32_t i) {
                if (i >= end) return -1;
                const int place = place_of(i), j = place - p.len;
                if (!known && place - lane + 32 > p.len) {
                    present = TreeWords(P, TreeParents(P, p.b, lane), lane).present();
                    known = true;
                }
                if (place >= p.n || (j >= 0 && !((present >> j) & 1ull))) return -1;
                const int page = table[place >> shift];
                return page < P.c.pages ? page : -1;
            };
            TokenRegs<D> r;
            int page = page_of(piece);
#pragma unroll 1
            for (bool begun = false; piece < end || !begun; begun = true) {
                // the record of this piece is decoded, the next one's loaded, the page of
                // the one after looked up (the first step only loads)
                if (begun) {
                    const uint32_t t = piece / kPieces, st = t & 1u;
                    const bool values = piece & 4u;
                    if (!a_mbar_wait_warp(bar((values ? kVEmpty : kKEmpty) + (int)st), ((t >> 1) & 1u) ^ 1u,
                                          P.timeout_cycles)) {
                        give_up();
                        break;
                    }
                    decode_token<D>(r, base + (values ? S::kV : S::kK) + st * S::kOperand,
                                    (int)(piece & 3u) * 32 + lane);
                    a_proxy_fence();
                    __syncwarp();
                    // (never, where a test wants the waits for it to run out)
                    if (lane == 0 && !(P.inject_skip && p.unit == 0 && p.ta == 0 && piece == tile_no * kPieces))
                        a_arrive(bar((values ? kVFull : kKFull) + (int)st));
                    piece += kDecodeWarps;
                }
                if (piece < end) {
                    const int64_t rec = (((int64_t)page * 2 * P.c.kv_heads + p.head) << shift) +
                                        (piece & 4u ? v_rows : 0) + (place_of(piece) & in_page);
                    load_token<D>(P, rec, page >= 0, r);
                }
                page = page_of(piece + kDecodeWarps);
            }
            tile_no = end / kPieces;
        }
    } else {
        // ---- tensor-core issue -----------------------------------------------------
        // The whole warp walks and waits, one elected lane issues: descriptors
        // stay warp-uniform that way (uniform registers are what the
        // instruction reads).  Broadcasts say so where values come from memory.
        uint32_t tile_no = 0, jobs_done[2] = {0, 0};  // before this part
        const bool elected = a_elect();
        const uint64_t q_desc = a_desc(base + S::kQ, 16), k_desc = a_desc(base + S::kK, 16);
        const uint64_t v_desc = a_desc(base + S::kV, S::kHalf);
        while (walk.next(P, p)) {
            a_named_sync(1, (kSoftWarps + 1) * 32);  // the queries are in place
            const int tiles = __shfl_sync(kFull, p.tb - p.ta, 0), jobs = pair ? 2 * tiles : tiles;
            auto score = [&](int i) {
                const uint32_t s = (uint32_t)i & 1u, t = tile_no + (uint32_t)(pair ? i >> 1 : i), st = t & 1u;
                // (the second stream of a pair finds the keys that the first waited for)
                if (!(pair && s) && !a_mbar_wait_warp(bar(kKFull + st), (t >> 1) & 1u, P.timeout_cycles)) {
                    give_up();
                    return;
                }
                a_fence_after();
                const uint64_t q = q_desc + (pair ? s : 0u) * (S::kOperand >> 4), k = k_desc + st * (S::kOperand >> 4);
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {  // 16 elements: 32 bytes along the swizzled row
                        const uint32_t o = ((uint32_t)(kk >> 2) * S::kHalf + 32u * (kk & 3)) >> 4;
                        a_mma_ss(128u * s, q + o, k + o, S::kIdescS, kk != 0);
                    }
                    a_commit(bar(kSFull + s));
                    if (!pair || s == 1) a_commit(bar(kKEmpty + st));
                }
                __syncwarp();
            };
            for (int i = 0; i < 2 && i < jobs && ok; ++i) score(i);
            for (int i = 0; i < jobs && ok; ++i) {
                const uint32_t s = (uint32_t)i & 1u, t = tile_no + (uint32_t)(pair ? i >> 1 : i), st = t & 1u;
                const uint32_t parity = ((s ? jobs_done[1] : jobs_done[0]) + (uint32_t)(i >> 1)) & 1u;
                if ((!(pair && s) && !a_mbar_wait_warp(bar(kVFull + st), (t >> 1) & 1u, P.timeout_cycles)) ||
                    !a_mbar_wait_warp(bar(kPReady + s), parity, P.timeout_cycles)) {
                    give_up();
                    break;
                }
                a_fence_after();
                const uint64_t v = v_desc + st * (S::kOperand >> 4);
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)  // 16 tokens: 8 columns of weights, 16 rows of V
                        a_mma_ts(kOCol + 128u * s, 128u * s + 8u * kk, v + 128u * kk, S::kIdescO, i >= 2 || kk != 0);
                    if (!pair || s == 1) a_commit(bar(kVEmpty + st));
                }
                __syncwarp();
                if (i + 2 < jobs) score(i + 2);
            }
            if (elected) a_commit(bar(kODone));  // all of this part's products
            __syncwarp();
            tile_no += (uint32_t)tiles;
            jobs_done[0] += (uint32_t)((jobs + 1) / 2);
            jobs_done[1] += (uint32_t)(jobs / 2);
            a_named_sync(1, (kSoftWarps + 1) * 32);  // results are read
        }
        if (!ok) {  // nothing may be in flight at the end; bounded like every wait
            if (elected) {
                a_commit(bar(kLast));
                a_mbar_wait(bar(kLast), 0u, P.timeout_cycles);
            }
            __syncwarp();
        }
    }
    // ---- teardown ---------------------------------------------------------------
    a_fence_before();
    __syncthreads();
    if (tid == 0) P.status[blockIdx.x] = *status;
    if (warp == kMmaWarp) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D>
cudaError_t launch_as(const AttnParams &P, cudaStream_t stream) {
    const cudaError_t e =
        cudaFuncSetAttribute(tc_attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcaShape<D>::kBytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(tc_attend_kernel<D>, P.workers, kTcaThreads, TcaShape<D>::kBytes, stream, P);
}

}  // namespace

bool tc_attention_fits(int head_dim) { return head_dim == 64 || head_dim == 128; }

int tc_attention_tile_rows(int rows) { return rows > kRowTile ? 2 * kRowTile : kRowTile; }

cudaError_t launch_tc_attention(const AttnParams &P, cudaStream_t stream) {
    return P.c.head_dim == 64 ? launch_as<64>(P, stream) : launch_as<128>(P, stream);
}

}  // namespace tq
