// tq_kv.cu -- the TQ4_1S key/value cache: rotary positions, quantising keys
// and values into the paged cache, reading them back, and moving an accepted
// branch's records together.
//
// A cache record is one token's head vector in the codec of the weights: per
// 32-element block the sign flip, the 32-point Walsh-Hadamard transform, two
// fp16 half-block scales and sixteen nibble codes per half (include/tq.h).
#include "tq_cache.cuh"
#include "tq_internal.h"

#include <algorithm>

namespace tq {

namespace {

__constant__ uint32_t c_kv_thr_bits[7] = TQ_THR_F32_INIT;
__constant__ uint32_t c_kv_mag_bits[8] = TQ_MAG_F32_INIT;

constexpr int kKvThreads = 256;

// One element as fp32, at any alignment of its own type.
template <int DT>
__device__ __forceinline__ float load1(const char *p) {
    if (DT == kF32) return *reinterpret_cast<const float *>(p);
    if (DT == kBF16) return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
    return __half2float(*reinterpret_cast<const __half *>(p));
}

// cos and sin of position * frequency, times `scale`.  The product of a 31-bit
// position and a 24-bit frequency is held in fp64 and reduced there to a
// fraction of a turn: in fp32 the angle of position 10^6 would be off by up
// to 0.03 rad.  What is left lies in [-1/2, 1/2] turns, where rounding it to
// fp32 costs at most 2^-25 turns.
__device__ __forceinline__ float2 rope_cos_sin(int position, float inv_freq, float scale, bool inverse) {
    constexpr double kPerTurn = 0.15915494309189533577;
    const double turns = (double)position * (double)inv_freq * kPerTurn;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    if (inverse) s = -s;
    return make_float2(c * scale, s * scale);
}

// ---------------------------------------------------------------------------
// Rotary positions.  A work item is V neighbouring pairs (or V elements past
// the rotated part) of one token for `hchunk` heads: the angles, which all
// heads share, are computed once per item.  Bound by HBM for long inputs
// (each element is read and written once), by the launch for one step.
// 8191 tokens x 32 heads x 128 in fp32, half of the elements rotated: 46.8 us,
// 5.7 TB/s; 64 tokens in bf16: 2.8 us.  Angle: 64-bit product and reduction to
// a turn, then 32-bit functions, so positions in the millions keep 2^-25 turns.
// ---------------------------------------------------------------------------
struct RopeParams {
    const char *x;
    char *out;
    const int32_t *positions;
    const float *inv_freq;
    int64_t x_token, x_head, o_token, o_head;  // strides in elements
    int64_t items;
    int heads, dim, rot, hchunk, chunks, slots, rot_slots;
    float scale;
    int interleaved, inverse, copy_tail;
};

// Heads whose loads go out together: the output may be the input, so the
// compiler cannot move a head's loads before another's stores by itself.  With
// eight pairs in a lane a second head costs more warps than it hides waits:
// 32768 tokens x 32 heads x 128 in bf16, one head 90 us and two 111 us; with
// four pairs (fp32), one head 98 us and four 89 us at 16384 tokens; element by
// element, 90 of 128 rotated, 92 and 75 us for 8192 tokens in fp32, 163 and 161
// for 16384 in bf16.
template <int V>
constexpr int kRopeAtOnce = V == 8 ? 1 : 4;

// V elements at p: one 16-byte access or a scalar one.
template <int DT, int V>
__device__ __forceinline__ void load_v(const char *p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = load1<DT>(p);
    } else if constexpr (DT == kF32) {
        const float4 q = *reinterpret_cast<const float4 *>(p);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (DT == kBF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

template <int DT, int V>
__device__ __forceinline__ void store_v(char *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        store1<DT>(p, v[0]);
    } else if constexpr (DT == kF32) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (DT == kBF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int DT, int V>
__global__ void __launch_bounds__(kKvThreads) rope_kernel(const RopeParams P) {
    constexpr int E = ElemSize<DT>::value, kRopeHeads = kRopeAtOnce<V>;
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t item = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
    if (item >= P.items) return;
    const int slot = (int)(item % P.slots);
    const int64_t rest = item / P.slots;
    const int chunk = (int)(rest % P.chunks);
    const int64_t token = rest / P.chunks;
    const int h0 = chunk * P.hchunk, h1 = min(P.heads, h0 + P.hchunk);
    const char *x = P.x + token * P.x_token * E;
    char *o = P.out + token * P.o_token * E;

    if (slot >= P.rot_slots) {  // past the rotated part: copied
        if (!P.copy_tail) return;
        const int e = P.rot + (slot - P.rot_slots) * V;
        for (int h = h0; h < h1; h += kRopeHeads) {
            float v[kRopeHeads][V];
#pragma unroll
            for (int k = 0; k < kRopeHeads; ++k)
                if (h + k < h1) load_v<DT, V>(x + ((h + k) * P.x_head + e) * E, v[k]);
#pragma unroll
            for (int k = 0; k < kRopeHeads; ++k)
                if (h + k < h1) store_v<DT, V>(o + ((h + k) * P.o_head + e) * E, v[k]);
        }
        return;
    }
    const int position = P.positions[token];
    float2 cs[V];
#pragma unroll
    for (int i = 0; i < V; ++i) cs[i] = rope_cos_sin(position, P.inv_freq[slot * V + i], P.scale, P.inverse);
    // pair i of the item: (a0 + i, a1 + i), or elements 2i, 2i+1 of 2V neighbours
    const int a0 = P.interleaved ? 2 * slot * V : slot * V;
    const int a1 = P.interleaved ? a0 + V : a0 + P.rot / 2;
    for (int h = h0; h < h1; h += kRopeHeads) {
        float u[kRopeHeads][V], w[kRopeHeads][V];
#pragma unroll
        for (int k = 0; k < kRopeHeads; ++k)
            if (h + k < h1) {
                load_v<DT, V>(x + ((h + k) * P.x_head + a0) * E, u[k]);
                load_v<DT, V>(x + ((h + k) * P.x_head + a1) * E, w[k]);
            }
#pragma unroll
        for (int k = 0; k < kRopeHeads; ++k) {
            float ru[V], rw[V];
            if (P.interleaved && V > 1) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 c0 = cs[i / 2], c1 = cs[(V + i) / 2];
                    ru[i] = u[k][i] * c0.x - u[k][i + 1] * c0.y;
                    ru[i + 1] = u[k][i] * c0.y + u[k][i + 1] * c0.x;
                    rw[i] = w[k][i] * c1.x - w[k][i + 1] * c1.y;
                    rw[i + 1] = w[k][i] * c1.y + w[k][i + 1] * c1.x;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    ru[i] = u[k][i] * cs[i].x - w[k][i] * cs[i].y;
                    rw[i] = u[k][i] * cs[i].y + w[k][i] * cs[i].x;
                }
            }
            if (h + k < h1) {
                store_v<DT, V>(o + ((h + k) * P.o_head + a0) * E, ru);
                store_v<DT, V>(o + ((h + k) * P.o_head + a1) * E, rw);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Cache addressing.
// ---------------------------------------------------------------------------
// Record of (page, plane, head, row), or -1 where the token has no place: a
// negative sequence or position, one past the table, or a page id outside the pool.
__device__ __forceinline__ int64_t record_page(const KvCache &C, int seq, int place) {
    if (seq < 0 || seq >= C.batch || place < 0) return -1;
    const int col = place >> C.page_shift;
    if (col >= C.pages_per_seq) return -1;
    const int64_t page = C.page_table[seq * C.table_ld + col];
    return page >= 0 && page < C.pages ? page : -1;
}

__device__ __forceinline__ int64_t record_index(const KvCache &C, int64_t page, int plane, int head, int place) {
    return (((page * 2 + plane) * C.kv_heads + head) << C.page_shift) + (place & ((1 << C.page_shift) - 1));
}

// ---------------------------------------------------------------------------
// Append: eight lanes own one 32-element block of one token (lane p elements
// 4p..4p+3) and walk `hchunk` heads of the key plane or of the value plane, so
// that a token's rotary angles are computed once for all of them.
// The arithmetic is tq_quantize's, operation for operation (butterfly stages
// 1, 2 in registers, 4, 8, 16 across lanes; adjacent-pair tree of squares).
// Bound by the launch and one item's chain: 64 tokens x 8 heads x 128 take
// 3.6 us with rotary positions, 2.9 without.
// ---------------------------------------------------------------------------
struct AppendParams {
    KvCache c;
    const char *x[2];
    int64_t token_stride[2], head_stride[2];  // elements
    const int32_t *seqs, *places;
    const int32_t *positions;  // null: no rotation
    const float *inv_freq;
    int64_t items;  // tokens * planes * chunks * blocks
    int rot, interleaved, blocks, hchunk, chunks;
    float scale;
};

// A half-block's code of y against its seven scaled thresholds.
__device__ __forceinline__ uint32_t cache_code(float y, const float (&t)[7]) {
    const float a = fabsf(y);
    const bool b2 = a > t[3];
    const bool b1 = a > (b2 ? t[5] : t[1]);
    const bool b0 = a > (b1 ? (b2 ? t[6] : t[2]) : (b2 ? t[4] : t[0]));
    return (b2 ? 4u : 0u) + (b1 ? 2u : 0u) + (b0 ? 1u : 0u) + (y < 0.0f ? 8u : 0u);
}

template <int DT>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const AppendParams P) {
    constexpr int E = ElemSize<DT>::value;
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t item = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) >> 3;
    const int p = threadIdx.x & 7;
    // lanes past the last item follow along without storing (the shuffles need whole warps)
    const int64_t it = item < P.items ? item : P.items - 1;
    const int block = (int)(it % P.blocks);
    int64_t rest = it / P.blocks;
    const int chunk = (int)(rest % P.chunks);
    rest /= P.chunks;
    const int plane = (int)(rest & 1);
    const int64_t token = rest >> 1;
    const int place = P.places[token];
    const int64_t page = record_page(P.c, P.seqs[token], place);
    const bool store = item < P.items && page >= 0;

    const int e0 = 32 * block + 4 * p;  // this lane's elements of the head
    uint32_t flips[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) flips[i] = sign_mask(e0 + i);
    float thr[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) thr[i] = __uint_as_float(c_kv_thr_bits[i]);

    // rotary partners: element e0 + i pairs with partner[i], its rotated value
    // is x cos + partner * (signed sin)
    const bool rotate = plane == 0 && P.positions != nullptr && e0 < P.rot;
    const int half = P.rot / 2;
    float2 cs[4];
    int first = 0;
    if (rotate) {
        const int position = P.positions[token];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + i;
            const bool lower = P.interleaved ? (e & 1) == 0 : e < half;
            const int pair = P.interleaved ? e >> 1 : (e < half ? e : e - half);
            cs[i] = e < P.rot ? rope_cos_sin(position, P.inv_freq[pair], P.scale, false) : make_float2(1.f, 0.f);
            if (lower) cs[i].y = -cs[i].y;
        }
        first = e0 < half ? e0 + half : e0 - half;
    }
    // the partners are four neighbours when the halves are split between lanes
    const bool whole = !P.interleaved && (half & 3) == 0 && (P.rot & 3) == 0;

    const char *base = P.x[plane] + token * P.token_stride[plane] * E;
    const int h0 = chunk * P.hchunk, h1 = min(P.c.kv_heads, h0 + P.hchunk);
    for (int h = h0; h < h1; ++h) {
        const char *x = base + (int64_t)h * P.head_stride[plane] * E;
        float v[4];
        load4_ordinary<DT>(x + e0 * E, v);
        if (rotate) {
            float o[4];
            if (P.interleaved) {
                o[0] = v[1]; o[1] = v[0]; o[2] = v[3]; o[3] = v[2];
            } else if (whole) {
                load4_ordinary<DT>(x + first * E, o);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = e0 + i;
                    o[i] = e < P.rot ? load1<DT>(x + (e < half ? e + half : e - half) * E) : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = v[i] * cs[i].x + o[i] * cs[i].y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = flip(v[i], flips[i]);
        fwht32_warp(v, p);

        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __fmul_rn(v[i], v[i]);
        float sum = __fadd_rn(__fadd_rn(q[0], q[1]), __fadd_rn(q[2], q[3]));
        sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, 1));
        sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, 2));
        // the scale saturates (and a NaN becomes the limit), so that every
        // record decodes to finite fp16 products c * d
        const __half hd = __float2half_rn(fminf(__fsqrt_rn(__fmul_rn(sum, 0.0625f)), kKvScaleMax));
        const float d = __half2float(hd);
        float t[7];
#pragma unroll
        for (int i = 0; i < 7; ++i) t[i] = __fmul_rn(thr[i], d);
        uint32_t code = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) code |= cache_code(v[i], t) << (4 * i);
        code |= __shfl_down_sync(kFull, code, 1) << 16;  // even lanes: eight codes
        const uint32_t dw = __half_as_ushort(hd);
        const uint32_t d2 = dw | (__shfl_down_sync(kFull, dw, 4) << 16);
        if (store) {
            const int64_t r = record_index(P.c, page, plane, h, place);
            if ((p & 1) == 0)
                *reinterpret_cast<uint32_t *>(P.c.codes + r * (P.c.head_dim / 2) + 16 * block + 2 * p) = code;
            if (p == 0) *reinterpret_cast<uint32_t *>(P.c.scales + r * (P.c.head_dim / 16) + 2 * block) = d2;
        }
    }
}

// ---------------------------------------------------------------------------
// Append, many tokens: a lane owns a whole block, the transform and the codes
// stay in its registers (no shuffles: 12 of them and a quarter of the sums are
// what the eight-lane form adds per four elements).  A CTA takes `per_cta`
// tokens; their rotary angles stand in shared memory, one fp64 reduction per
// token and pair.  Keys and values run one after the other, so that a warp's
// lanes agree about the rotation.
// Bound by the codec's arithmetic: 36 instructions an element, issue slots 67%
// used, ALU pipe 64%, FMA pipe 28%: the load on one pipe, not a limit reached.
// 16384 tokens x 8 heads x 128 in bf16 with rotary positions 49 us, 1.8 TB/s
// (without 41; with eight lanes a block 85).
// ---------------------------------------------------------------------------
constexpr int kAngles = 2048;  // cos, sin pairs of a CTA

// 32 elements as they are in memory, and as fp32.
template <int DT>
struct RawBlock {
    static constexpr int N = 2 * ElemSize<DT>::value;
    uint4 q[N];
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = ld(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ float at(int e) const {  // (e is a constant after unrolling)
        const uint4 &w4 = q[e * ElemSize<DT>::value / 16];
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
        if (DT == kF32) return __uint_as_float(w[e & 3]);
        const uint32_t x = w[(e >> 1) & 3];
        if (DT == kBF16) return __uint_as_float((e & 1) ? x & 0xffff0000u : x << 16);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
        return (e & 1) ? f.y : f.x;
    }
};

// v rotated in place; block `blk` of the head at `x`, angles of its token at cs.
template <int DT>
__device__ __forceinline__ void rotate_block(const AppendParams &P, const char *x, int blk, const float2 *cs,
                                             float (&v)[32]) {
    const int e0 = 32 * blk, half = P.rot / 2;
    if (P.interleaved) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 c = cs[(e0 + i) / 2];
            const float a = v[i] * c.x - v[i + 1] * c.y, b = v[i + 1] * c.x + v[i] * c.y;
            v[i] = a;
            v[i + 1] = b;
        }
        return;
    }
    const bool lower = e0 < half;
    RawBlock<DT> raw;
    raw.load(x + (lower ? e0 + half : e0 - half) * ElemSize<DT>::value);
    const float4 *c4 = reinterpret_cast<const float4 *>(cs + (lower ? e0 : e0 - half));
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float o[4] = {raw.at(i), raw.at(i + 1), raw.at(i + 2), raw.at(i + 3)};
        const float4 c0 = c4[i / 2], c1 = c4[i / 2 + 1];
        const float c[4] = {c0.x, c0.z, c1.x, c1.z}, sn[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[i + k] = v[i + k] * c[k] + o[k] * (lower ? -sn[k] : sn[k]);
    }
}

template <int DT>
__global__ void __launch_bounds__(kKvThreads, DT == kF32 ? 2 : 3)
    kv_append_block_kernel(const AppendParams P, int per_cta) {
    constexpr int E = ElemSize<DT>::value;
    __shared__ __align__(16) float2 angles[kAngles];
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t token0 = (int64_t)blockIdx.x * per_cta;
    const int tokens = (int)min((int64_t)per_cta, P.items - token0);
    const int pairs = P.rot / 2;
    if (P.positions) {
        for (int i = threadIdx.x; i < tokens * pairs; i += kKvThreads)
            angles[i] = rope_cos_sin(P.positions[token0 + i / pairs], P.inv_freq[i % pairs], P.scale, false);
        __syncthreads();
    }
    float thr[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) thr[i] = __uint_as_float(c_kv_thr_bits[i]);
    const int per_plane = P.c.kv_heads * P.blocks;
    for (int plane = 0; plane < 2; ++plane) {
        for (int i = threadIdx.x; i < tokens * per_plane; i += kKvThreads) {
            const int t = i / per_plane, rest = i - t * per_plane;
            const int head = rest / P.blocks, blk = rest - head * P.blocks;
            const int64_t token = token0 + t;
            const char *x = P.x[plane] + (token * P.token_stride[plane] + head * P.head_stride[plane]) * E;
            RawBlock<DT> raw;
            raw.load(x + 32 * blk * E);
            const int place = P.places[token];
            const int64_t page = record_page(P.c, P.seqs[token], place);
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = raw.at(e);
            if (plane == 0 && P.positions && 32 * blk < P.rot) rotate_block<DT>(P, x, blk, angles + t * pairs, v);
            const uint32_t bits = c_sign_words.w[blk];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = flip(v[e], (bits << (31 - e)) & 0x80000000u);
            fwht32_regs(v);
            uint32_t dbits[2];
            float D[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float q[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) q[e] = __fmul_rn(v[16 * h + e], v[16 * h + e]);
#pragma unroll
                for (int step = 1; step < 16; step <<= 1)
#pragma unroll
                    for (int e = 0; e < 16; e += 2 * step) q[e] = __fadd_rn(q[e], q[e + step]);
                const __half hd = __float2half_rn(fminf(__fsqrt_rn(__fmul_rn(q[0], 0.0625f)), kKvScaleMax));
                dbits[h] = __half_as_ushort(hd);
                D[h] = __half2float(hd);
            }
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float lim[7];
#pragma unroll
                for (int k = 0; k < 7; ++k) lim[k] = __fmul_rn(thr[k], D[h]);
#pragma unroll
                for (int e = 16 * h; e < 16 * h + 16; ++e) w[e >> 3] = add_code(w[e >> 3], v[e], lim, 4 * (e & 7));
            }
            if (page >= 0) {
                const int64_t r = record_index(P.c, page, plane, head, place);
                *reinterpret_cast<uint4 *>(P.c.codes + r * (P.c.head_dim / 2) + 16 * blk) =
                    make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint32_t *>(P.c.scales + r * (P.c.head_dim / 16) + 2 * blk) =
                    dbits[0] | (dbits[1] << 16);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Read: the eight-lane layout in reverse.  x~ = s . (H (c d)) / 32 in fp32
// (tq_dequantize's order), rounded once to the output type.
// ---------------------------------------------------------------------------
struct ReadParams {
    KvCache c;
    char *out[2];
    int64_t token_stride[2], head_stride[2];
    const int32_t *seqs, *places;
    int64_t items;
    int blocks, hchunk, chunks;
};

template <int DT>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const ReadParams P) {
    constexpr int E = ElemSize<DT>::value;
    // sixteen signed centroids, one bank each: any mix of codes in a warp is
    // one conflict-free access
    __shared__ float table[16];
    if (threadIdx.x < 16)
        table[threadIdx.x] = __uint_as_float(c_kv_mag_bits[threadIdx.x & 7] ^ ((threadIdx.x & 8u) << 28));
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();
    const int64_t item = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) >> 3;
    const int p = threadIdx.x & 7;
    const int64_t it = item < P.items ? item : P.items - 1;
    const int block = (int)(it % P.blocks);
    int64_t rest = it / P.blocks;
    const int chunk = (int)(rest % P.chunks);
    rest /= P.chunks;
    const int plane = (int)(rest & 1);
    const int64_t token = rest >> 1;
    const int place = P.places[token];
    const int64_t page = record_page(P.c, P.seqs[token], place);
    const int e0 = 32 * block + 4 * p;
    uint32_t flips[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) flips[i] = sign_mask(e0 + i);
    char *base = P.out[plane] + token * P.token_stride[plane] * E;
    const int h0 = chunk * P.hchunk, h1 = min(P.c.kv_heads, h0 + P.hchunk);
    for (int h = h0; h < h1; ++h) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (page >= 0) {
            const int64_t r = record_index(P.c, page, plane, h, place);
            const uint32_t w =
                *reinterpret_cast<const uint16_t *>(P.c.codes + r * (P.c.head_dim / 2) + 16 * block + 2 * p);
            const float d = __fmul_rn(
                __half2float(__ushort_as_half(P.c.scales[r * (P.c.head_dim / 16) + 2 * block + (p >> 2)])), 0.03125f);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(table[(w >> (4 * i)) & 15u], d);
        }
        fwht32_warp(v, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = flip(v[i], flips[i]);
        if (item < P.items) store4<DT>(base + ((int64_t)h * P.head_stride[plane] + e0) * E, v);
    }
}

// Read, many tokens: a lane owns a block; a warp's 32 blocks leave through a
// stage in shared memory (16-byte chunks, XOR-placed against bank conflicts), so
// that stores cover whole head vectors instead of 64-byte pieces.  16384 tokens
// x 8 heads x 128 to bf16: 27 us, 3.2 TB/s, issue slots 68% used (eight lanes a
// block: 49 us).
template <int DT>
__global__ void __launch_bounds__(kKvThreads, DT == kF32 ? 2 : 3) kv_read_block_kernel(const ReadParams P) {
    constexpr int E = ElemSize<DT>::value, C = 2 * E;  // 16-byte chunks of a block
    __shared__ float table[16];
    __shared__ __align__(16) uint4 stage[kKvThreads * C];
    if (threadIdx.x < 16)
        table[threadIdx.x] = __uint_as_float(c_kv_mag_bits[threadIdx.x & 7] ^ ((threadIdx.x & 8u) << 28));
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();
    const int lane = threadIdx.x & 31;
    uint4 *st = stage + (threadIdx.x & ~31) * C;
    auto key = [](int l) { return C == 8 ? (l & 7) : ((l >> 1) & 3); };
    // blocks in the order token, plane, head, block of the head; this lane's one
    const int64_t first = ((int64_t)blockIdx.x * kKvThreads + threadIdx.x) - lane;
    if (first >= P.items) return;
    const int per_token = 2 * P.c.kv_heads * P.blocks;
    const int64_t i = min(first + lane, P.items - 1);
    const int64_t token = quotient(i, per_token);
    const int rest = (int)(i - token * per_token);
    const int plane_head = rest / P.blocks, blk = rest - plane_head * P.blocks;
    const int plane = plane_head >= P.c.kv_heads, head = plane_head - plane * P.c.kv_heads;
    char *mine = P.out[plane] + (token * P.token_stride[plane] + head * P.head_stride[plane] + 32 * blk) * E;
    {
        const int place = P.places[token];
        const int64_t page = record_page(P.c, P.seqs[token], place);
        float v[32];
        if (page >= 0) {
            const int64_t r = record_index(P.c, page, plane, head, place);
            const uint4 w4 = *reinterpret_cast<const uint4 *>(P.c.codes + r * (P.c.head_dim / 2) + 16 * blk);
            const uint32_t sc = *reinterpret_cast<const uint32_t *>(P.c.scales + r * (P.c.head_dim / 16) + 2 * blk);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            const float2 D = __half22float2(*reinterpret_cast<const __half2 *>(&sc));
            const float Ds[2] = {__fmul_rn(D.x, 0.03125f), __fmul_rn(D.y, 0.03125f)};
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __fmul_rn(table[(w[e >> 3] >> (4 * (e & 7))) & 15u], Ds[e >> 4]);
            fwht32_regs(v);
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
        // rounded, signs put on the rounded values
        const uint32_t signs = DT == kF32 ? c_sign_words.w[blk] : c_sign_pairs.w[blk];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (DT == kF32) {
                    o[k] = __float_as_uint(v[4 * c + k]) ^ ((signs << (31 - 4 * c - k)) & 0x80000000u);
                } else {
                    const int p = (4 * c + k) % 16;  // pair
                    if (DT == kBF16) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * p], v[2 * p + 1]);
                        o[k] = *reinterpret_cast<const uint32_t *>(&h);
                    } else {
                        const __half2 h = __floats2half2_rn(v[2 * p], v[2 * p + 1]);
                        o[k] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    o[k] ^= (signs << (15 - p)) & 0x80008000u;
                }
            }
            st[lane * C + (c ^ key(lane))] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    __syncwarp();
#pragma unroll
    for (int c0 = 0; c0 < C; ++c0) {
        const int c = c0 * 32 + lane, l = c / C;
        char *dst = reinterpret_cast<char *>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(mine), l));
        if (first + l < P.items)
            *reinterpret_cast<uint4 *>(dst + 16 * (c % C)) = st[l * C + ((c % C) ^ key(l))];
    }
}

// ---------------------------------------------------------------------------
// Commit: the records of an accepted branch move down to where the sequence
// continues.  A CTA takes one layer of one sequence: its first warp finds the
// branch's records, once for all planes, heads and pieces; then a thread owns a
// 16-byte piece of the codes (or 4 bytes of the scales) of a (plane, head) and
// moves it for the whole branch, eight records at a time, all eight loads
// before the stores.  The branch increases, so a record's target never lies
// behind a source that is still to be read.  Bound by two rounds of dependent
// loads (path and page ids, then records): 32 layers x one sequence 4.1 us, 32
// layers x 64 sequences of 8 heads x 128, eight accepted of 64, 12.6 us.
// ---------------------------------------------------------------------------
struct CommitParams {
    KvCache c;  // of layer 0
    int64_t code_layer, scale_layer;  // strides of a layer, elements
    const int32_t *lens, *path;
    int64_t path_ld;
    int steps, pieces, code_pieces;
};
constexpr int kMaxSteps = 64;

// Moves piece (plane_head, offset) of the branch's records; `from` and `to` are
// the rows of plane 0, head 0 (to < 0: nothing to move).
template <typename T>
__device__ __forceinline__ void move_branch(char *pool, const int64_t *from, const int64_t *to, int count,
                                            int64_t row, int64_t record_bytes, int offset) {
    for (int i0 = 0; i0 < count; i0 += 8) {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i < count && to[i0 + i] >= 0)
                v[i] = *reinterpret_cast<const T *>(pool + (from[i0 + i] + row) * record_bytes + offset);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i0 + i < count && to[i0 + i] >= 0)
                *reinterpret_cast<T *>(pool + (to[i0 + i] + row) * record_bytes + offset) = v[i];
    }
}

__global__ void __launch_bounds__(kKvThreads) kv_commit_kernel(const CommitParams P) {
    __shared__ int64_t from[kMaxSteps], to[kMaxSteps];
    __shared__ int branch;
    grid_dependency_wait();
    grid_dependents_launch();
    const int seq = blockIdx.x % P.c.batch, lane = threadIdx.x & 31;
    const int64_t layer = blockIdx.x / P.c.batch;
    if (threadIdx.x < 32) {
        const int len = max(P.lens[seq], 0);
        const int32_t *path = P.path + seq * P.path_ld;
        uint32_t ends[2];
        int src[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = lane + 32 * k;
            src[k] = i < P.steps ? path[i] : -1;
            const int before = i > 0 && i < P.steps ? path[i - 1] : -1;
            ends[k] = __ballot_sync(kFull, i >= P.steps || src[k] <= before || src[k] > INT32_MAX - len);
        }
        const int count = ends[0] ? __ffs(ends[0]) - 1 : ends[1] ? 31 + __ffs(ends[1]) : 64;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = lane + 32 * k;
            if (i >= count) continue;
            const int64_t a = record_page(P.c, seq, len + src[k]), z = record_page(P.c, seq, len + i);
            const bool moves = src[k] != i && a >= 0 && z >= 0;
            from[i] = moves ? record_index(P.c, a, 0, 0, len + src[k]) : -1;
            to[i] = moves ? record_index(P.c, z, 0, 0, len + i) : -1;
        }
        if (lane == 0) branch = count;
    }
    __syncthreads();
    const int count = branch;
    for (int item = threadIdx.x; item < 2 * P.c.kv_heads * P.pieces; item += blockDim.x) {
        const int plane_head = item / P.pieces, piece = item - plane_head * P.pieces;
        const int64_t row = (int64_t)plane_head << P.c.page_shift;
        if (piece < P.code_pieces)
            move_branch<uint4>(reinterpret_cast<char *>(P.c.codes + layer * P.code_layer), from, to, count, row,
                               P.c.head_dim / 2, 16 * piece);
        else
            move_branch<uint32_t>(reinterpret_cast<char *>(P.c.scales + layer * P.scale_layer), from, to, count, row,
                                  P.c.head_dim / 8, 4 * (piece - P.code_pieces));
    }
}

// Heads per work item, which share its angles and indices: up to eight while
// the launch still has kEnoughThreads (three or four warps for each of the
// GPU's 592 schedulers); short inputs take one head per item.  Rotary positions
// of 32 heads x 128 in bf16: 512 tokens 4.1 us, 5.3 us where 2^18 threads are
// enough; 2048 tokens 7.6 and 8.7; at most 4, 8 and all heads, 8192 tokens
// 26.9, 28.2 and 36.1 us; 32768 tokens 91.5, 89.7 and 98.7; of 8191 tokens in
// fp32 with half of the elements rotated 50.4, 46.8 and 47.2.
constexpr int64_t kEnoughThreads = 1 << 16;
constexpr int kMostHeads = 8;

int heads_per_item(int64_t threads_per_head, int heads) {
    int h = std::min(heads, kMostHeads);
    for (; h > 1; --h) {
        const int64_t threads = threads_per_head * ((heads + h - 1) / h);
        // in a launch of one wave the longest item decides: equal shares
        if (threads >= (heads % h ? 4 * kEnoughThreads : kEnoughThreads)) break;
    }
    return h;
}

// Blocks from which on a lane takes a whole one; below, eight lanes share a
// block and finish sooner.  Append of bf16 with rotary positions, 8 heads x 128,
// eight lanes against one: 2^14 blocks 4.6 and 6.5 us, 2^15 blocks 6.6 and 6.6,
// 2^16 blocks 9.7 and 6.7, 2^20 blocks 85 and 50.  Read: 2^14 blocks 3.3 and
// 3.1, 2^15 blocks 4.5 and 3.1, 2^20 blocks 49 and 27.  (One bound for both: the
// read alone could turn a power of two lower.)
constexpr int64_t kManyBlocks = 1 << 15;

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + kKvThreads - 1) / kKvThreads); }

}  // namespace

cudaError_t launch_rope(const RopeJob &j, cudaStream_t stream) {
    const int esize = j.dtype == kF32 ? 4 : 2, vec = 16 / esize;
    // whole 16-byte accesses where every part and stride allows them; else
    // element by element: 16384 tokens x 32 heads x 128 in bf16, all rotated 48
    // us, 90 of 128 rotated 161 us; 8192 tokens in fp32 43 and 75 us
    const bool wide = j.rot % (2 * vec) == 0 && j.dim % vec == 0 && j.x_token % vec == 0 && j.x_head % vec == 0 &&
                      j.o_token % vec == 0 && j.o_head % vec == 0 && reinterpret_cast<uintptr_t>(j.x) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(j.out) % 16 == 0;
    const int V = wide ? vec : 1;
    RopeParams P;
    P.x = static_cast<const char *>(j.x);
    P.out = static_cast<char *>(j.out);
    P.positions = j.positions;
    P.inv_freq = j.inv_freq;
    P.x_token = j.x_token;
    P.x_head = j.x_head;
    P.o_token = j.o_token;
    P.o_head = j.o_head;
    P.heads = j.heads;
    P.dim = j.dim;
    P.rot = j.rot;
    P.scale = j.scale;
    P.interleaved = j.interleaved;
    P.inverse = j.inverse;
    P.copy_tail = j.out != j.x;
    P.rot_slots = j.rot / 2 / V;
    P.slots = P.rot_slots + (P.copy_tail ? (j.dim - j.rot) / V : 0);
    if (P.slots == 0) return cudaSuccess;
    P.hchunk = heads_per_item(j.tokens * P.slots, j.heads);
    P.chunks = (j.heads + P.hchunk - 1) / P.hchunk;
    P.items = j.tokens * P.chunks * P.slots;
    const unsigned grid = blocks_of(P.items);
    cudaError_t e = cudaSuccess;
    auto run = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        constexpr int W = 16 / ElemSize<DT>::value;
        if (wide) e = launch_dependent(rope_kernel<DT, W>, grid, kKvThreads, 0, stream, P);
        else e = launch_dependent(rope_kernel<DT, 1>, grid, kKvThreads, 0, stream, P);
    };
    if (j.dtype == kF32) run(std::integral_constant<int, kF32>());
    else if (j.dtype == kBF16) run(std::integral_constant<int, kBF16>());
    else run(std::integral_constant<int, kF16>());
    return e;
}

cudaError_t launch_kv_append(const KvAppendJob &j, cudaStream_t stream) {
    AppendParams P;
    P.c = j.c;
    for (int i = 0; i < 2; ++i) {
        P.x[i] = static_cast<const char *>(j.x[i]);
        P.token_stride[i] = j.token_stride[i];
        P.head_stride[i] = j.head_stride[i];
    }
    P.seqs = j.seqs;
    P.places = j.places;
    P.positions = j.positions;
    P.inv_freq = j.inv_freq;
    P.rot = j.rot;
    P.interleaved = j.interleaved;
    P.scale = j.scale;
    P.blocks = j.c.head_dim / 32;
    // whole blocks per lane once there are enough of them, and where a block's
    // rotary partners are a block too: 16384 tokens x 8 heads in bf16, 64 of 96
    // rotated 42 us, all of 96 (halves of 48) with eight lanes a block 78; of 128,
    // 64, 96 and 128 rotated 49, 92 and 51 us
    const bool whole = !j.positions || (j.rot % 32 == 0 && (j.interleaved || j.rot % 64 == 0));
    if (j.tokens * 2 * j.c.kv_heads * P.blocks >= kManyBlocks && whole) {
        const int64_t of_token = j.c.kv_heads * P.blocks;  // blocks of a plane
        int64_t per = of_token >= kKvThreads ? 1 : kKvThreads / of_token;
        if (j.positions && per * (j.rot / 2) > kAngles) per = kAngles / (j.rot / 2);
        P.items = j.tokens;
        const unsigned grid = (unsigned)((j.tokens + per - 1) / per);
        if (j.dtype == kF32)
            return launch_dependent(kv_append_block_kernel<kF32>, grid, kKvThreads, 0, stream, P, (int)per);
        if (j.dtype == kBF16)
            return launch_dependent(kv_append_block_kernel<kBF16>, grid, kKvThreads, 0, stream, P, (int)per);
        return launch_dependent(kv_append_block_kernel<kF16>, grid, kKvThreads, 0, stream, P, (int)per);
    }
    P.hchunk = heads_per_item(j.tokens * 2 * P.blocks * 8, j.c.kv_heads);
    P.chunks = (j.c.kv_heads + P.hchunk - 1) / P.hchunk;
    P.items = j.tokens * 2 * P.chunks * P.blocks;
    const unsigned grid = blocks_of(P.items * 8);
    cudaError_t e;
    if (j.dtype == kF32) e = launch_dependent(kv_append_kernel<kF32>, grid, kKvThreads, 0, stream, P);
    else if (j.dtype == kBF16) e = launch_dependent(kv_append_kernel<kBF16>, grid, kKvThreads, 0, stream, P);
    else e = launch_dependent(kv_append_kernel<kF16>, grid, kKvThreads, 0, stream, P);
    return e;
}

cudaError_t launch_kv_read(const KvReadJob &j, cudaStream_t stream) {
    ReadParams P;
    P.c = j.c;
    for (int i = 0; i < 2; ++i) {
        P.out[i] = static_cast<char *>(j.out[i]);
        P.token_stride[i] = j.token_stride[i];
        P.head_stride[i] = j.head_stride[i];
    }
    P.seqs = j.seqs;
    P.places = j.places;
    P.blocks = j.c.head_dim / 32;
    P.items = j.tokens * 2 * j.c.kv_heads * P.blocks;
    if (P.items >= kManyBlocks) {
        const unsigned grid = blocks_of(P.items);
        if (j.dtype == kF32) return launch_dependent(kv_read_block_kernel<kF32>, grid, kKvThreads, 0, stream, P);
        if (j.dtype == kBF16) return launch_dependent(kv_read_block_kernel<kBF16>, grid, kKvThreads, 0, stream, P);
        return launch_dependent(kv_read_block_kernel<kF16>, grid, kKvThreads, 0, stream, P);
    }
    P.hchunk = heads_per_item(j.tokens * 2 * P.blocks * 8, j.c.kv_heads);
    P.chunks = (j.c.kv_heads + P.hchunk - 1) / P.hchunk;
    P.items = j.tokens * 2 * P.chunks * P.blocks;
    const unsigned grid = blocks_of(P.items * 8);
    cudaError_t e;
    if (j.dtype == kF32) e = launch_dependent(kv_read_kernel<kF32>, grid, kKvThreads, 0, stream, P);
    else if (j.dtype == kBF16) e = launch_dependent(kv_read_kernel<kBF16>, grid, kKvThreads, 0, stream, P);
    else e = launch_dependent(kv_read_kernel<kF16>, grid, kKvThreads, 0, stream, P);
    return e;
}

cudaError_t launch_kv_commit(const KvCommitJob &j, cudaStream_t stream) {
    CommitParams P;
    P.c = j.c;
    P.code_layer = j.code_layer;
    P.scale_layer = j.scale_layer;
    P.lens = j.lens;
    P.path = j.path;
    P.path_ld = j.path_ld;
    P.steps = j.steps;
    P.code_pieces = j.c.head_dim / 32;
    P.pieces = P.code_pieces + j.c.head_dim / 32;
    // (a CTA no wider than a layer's pieces need)
    const int pieces = 2 * j.c.kv_heads * P.pieces;
    const unsigned threads = pieces >= kKvThreads ? kKvThreads : (unsigned)(pieces + 31) / 32 * 32;
    return launch_dependent(kv_commit_kernel, (unsigned)(j.layers * j.c.batch), threads, 0, stream, P);
}

}  // namespace tq
