// tq_attention.cu -- attention of drafted tokens over the TQ4_1S cache.
//
// Mathematics.  With H the 32-point Hadamard matrix and s the codec's signs, a
// cached vector is k~ = s . (H (c d)) / 32 per 32-element block, so
//   q . k~ = sum_e (H (s . q) / 32)_e c_e d_h(e)
// and a weighted sum of values is
//   sum_j p_j v~_j = s . (H (sum_j p_j c_j d_j)) / 32:
// the query is rotated once, the result is rotated back once, and a cached
// token costs a table lookup and a scale per element.  The softmax runs in
// one pass over the tokens with a running maximum and sum (both fp32).
//
// attend_kernel (mma.sync, tiles of 8 or 16 rows).  The groups of 16 tokens of
// all units are cut into equal ranges, one per warp, and a warp works alone: no
// barrier, no exchange but shuffles, so that one warp's wait for a unit's first
// loads is hidden by the others.  Per group:
//   S^T [16 tokens x 8 rows] = K [16 x D] q^T      (tokens on the M side, so
//   O^T [D x 8 rows] += V^T [D x 16] P^T            no row of the product is padding)
// A byte of codes (two elements) is turned into a pair of fp16 centroids by one
// lookup in a shared-memory table with a column for each lane, so that lookups
// never meet in a bank: 256 rows of 128 bytes, 256 bytes apart, on a 64 KB
// boundary, which makes the address (code byte, lane) a single byte permute.
// Per pair: one PRMT, one LDS, one HMUL2 by the half-block's scale.  The values'
// pairs have to hold two tokens of one element; nibbles of two tokens' code
// words are merged before the lookup (two operations per 8 codes).
// Roundings to fp16: centroid (2^-12 relative), centroid x scale, rotated
// query (as in the products of this library; times the softmax's scale and a
// power of two, RowScale), and the softmax weights, which are scaled by 2^7.
// The maximum they refer to is followed only when it grows by more than 2^8
// (rescaling the accumulators is the exception), so a weight is at most 2^15,
// and weights down to 2^-31 of the largest survive.
//
// What bounds it: instruction issue and shared-memory lookups, not HBM.  Per
// pair of elements of a group the lookup, its address and the scale are three
// instructions whatever the rows, so up to 8 rows cost the same.  64 sequences,
// 289,000 tokens together, 32 query over 8 key/value heads of 128: 97.5 us with
// the joining launch, 3.8 TB/s of records (issue slots 60% used, the
// shared-memory pipe 56%); 96.2 before rows had a power of two of their own,
// which takes two registers.  One sequence of 1000 tokens 11.6 us, of 4000 16.5,
// of 30000 28: two launches, a warp's chain of waits (page id, records, query),
// hence ranges down to one group, so that many warps share few tokens; and a
// part of every warp (up to 297 a row) that the joining launch has to read.
#include "tq_attention.cuh"

namespace tq {

namespace {

constexpr int kGroup = 16;               // tokens of a group
constexpr uint32_t kLutBase = 0x10000u;  // shared-memory address of the centroid table
constexpr uint32_t kLutStep = 256;       // bytes between its rows (128 used)
// Groups of a warp's range at least: a single token over 1000 cached ones takes
// 11.6 us with 1 and 12.1 with 4.  (Over 4000 16.5 and 12.5: there fewer parts
// weigh more.)
constexpr int kLeastGroups = 1;
// What beginning a unit costs (its query rotated, its part written), in groups:
// 0, 2, 4 and 8 take 98.8, 97.3, 96.9 and 97.6 us for 64 sequences of up to 8000
// tokens; in tiles of the tcgen05 kernel, 0, 2, 3, 4 and 5 take 63.8, 55.2, 52.8,
// 51.5 and 51.4 us for 16 trees of 16 tokens and 162.7, 160.6, 158.6, 158.1 and
// 156.2 us for 4 trees of 64.
constexpr int kExtraGroups = 4;
constexpr int kTcExtra = 4;
// Rows of a key/value head above which the tcgen05 kernel runs.  mma.sync
// against tcgen05, head dimension 128: 16 sequences of 4000 tokens with 16 rows
// 46 and 64 us, with 24 rows 69 and 65; 4 of 30000 tokens 68 and 98, 115 and 99.
constexpr int kTcLeastRows = 16;

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pair of centroids of byte `B` of w (low nibble in the low half).
template <int B>
__device__ __forceinline__ uint32_t lut_pair(uint32_t w, uint32_t lane_base) {
    uint32_t v;
    // address bytes: lane * 4, code byte, 0x01 and 0x00 of the table's base
    const uint32_t a = prmt(lane_base, w, 0x3200u | ((4u + B) << 4));
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ void fill_lut(int tid, int threads) {
    for (int i = tid; i < 256 * 8; i += threads) {
        uint32_t o[4];
        decode_word((uint32_t)(i >> 3), o);
        const uint32_t a = kLutBase + (uint32_t)(i >> 3) * kLutStep + (uint32_t)(i & 7) * 16;
        asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(o[0]) : "memory");
    }
}

// The rotated query as operand fragments, straight from memory: lane
// l = 4 g + c owns row g, elements DP/4 c .. of it, which for a head dimension
// of 128 is one whole block (of 64: half of one, the other half at lane ^ 1),
// so that the transform runs in registers.  `x` is the lane's row.  Returns the
// unit of row g's scores.
template <int DT, int DP>
__device__ __forceinline__ float rotate_query(const AttnParams &P, const char *x, bool valid, int c,
                                              uint32_t (&qf)[DP / 16][2]) {
    constexpr int N = DP / 4 < 32 ? 16 : 32;  // elements of a block that the lane holds
    constexpr int B = DP / 4 / N;             // such pieces
    float v[B][N], most[2] = {0.f, 0.f};
#pragma unroll
    for (int blk = 0; blk < B; ++blk) {
        const int e0 = c * (DP / 4) + blk * N;
        const uint32_t bits = c_sign_words.w[e0 / 32] >> (e0 % 32);
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            if (valid && e0 < P.c.head_dim) load4_ordinary<DT>(x + (int64_t)(e0 + i) * ElemSize<DT>::value, t);
#pragma unroll
            for (int k = 0; k < 4; ++k) most[k & 1] = fmaxf(most[k & 1], fabsf(t[k]));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[blk][i + k] = flip(t[k], (bits << (31 - i - k)) & 0x80000000u);
        }
    }
    float all = fmaxf(most[0], most[1]);
    all = fmaxf(all, __shfl_xor_sync(kFull, all, 1));
    all = fmaxf(all, __shfl_xor_sync(kFull, all, 2));
    const RowScale scale(P.q_factor, all);
#pragma unroll
    for (int blk = 0; blk < B; ++blk) {
#pragma unroll
        for (int h = 1; h < N; h <<= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((i & h) == 0) {
                    const float a = v[blk][i], b = v[blk][i + h];
                    v[blk][i] = a + b;
                    v[blk][i + h] = a - b;
                }
        if (N == 16) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[blk][i] = butterfly_xlane(v[blk][i], 1, c & 1);
        }
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const __half2 h = __floats2half2_rn(v[blk][i] * scale.factor, v[blk][i + 1] * scale.factor);
            qf[(blk * N + i) / 4][(i / 2) & 1] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return scale.unit;
}

// What a lane (l = 4 g + c) holds of a group of 16 tokens.  Key rows: tokens
// g / 2 + 4 (g % 2) and that + 8, elements DP/4 * c ...; value rows: tokens
// c, c + 4, c + 8, c + 12, elements DP/8 * g ...  In this order S^T's accumulator,
// transposed by movmatrix, is the weights operand of the second product, and
// every load of the warp covers whole neighbouring rows.
template <int DP>
struct KeyRegs {
    static constexpr int W = DP / 32;  // code words of a row (DP / 4 elements)
    static constexpr int D = DP / 64;  // its half-block scales
    uint32_t w[2][W];
    uint32_t d[2][(D + 1) / 2];
};
template <int DP>
struct ValueRegs {
    static constexpr int W = DP / 64;  // code words of a row (DP / 8 elements)
    static constexpr int H = DP < 256 ? 1 : 2;
    uint32_t w[4][W];
    uint32_t d[4];  // one or two half-block scales
};

// Where this lane's rows begin within a group (added to warp-uniform bases);
// with FULL the head dimension is DP itself and no piece is missing.
template <int DP, bool FULL>
struct LaneOffsets {
    int dim;
    uint32_t kc, ks, vc, vs;  // bytes
    __device__ __forceinline__ LaneOffsets(int head_dim, int lane) {
        const int g = lane >> 2, c = lane & 3;
        dim = FULL ? DP : head_dim;
        const int row = (g >> 1) + 4 * (g & 1);
        kc = row * (dim / 2) + c * (DP / 8);
        ks = row * (dim / 8) + c * (DP / 32);
        vc = c * (dim / 2) + g * (DP / 16);
        vs = c * (dim / 8) + g * (DP / 8) / 16 * 2;
    }
};

template <int DP, bool FULL>
__device__ __forceinline__ void load_keys(const uint8_t *codes, const uint8_t *scales,
                                          const LaneOffsets<DP, FULL> &o, int c, KeyRegs<DP> &r) {
    const int dim = FULL ? DP : o.dim;
    codes += o.kc;
    scales += o.ks;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint8_t *cp = codes + i * 4 * dim;  // eight rows on
        const uint8_t *sp = scales + i * dim;
        if constexpr (DP == 64) {
            uint2 w = make_uint2(0u, 0u);
            uint32_t d = 0;
            if (FULL || 16 * c < dim) {
                w = ld(reinterpret_cast<const uint2 *>(cp));
                d = ld(reinterpret_cast<const uint16_t *>(sp));
            }
            r.w[i][0] = w.x;
            r.w[i][1] = w.y;
            r.d[i][0] = d;
        } else {
#pragma unroll
            for (int j = 0; j < DP / 128; ++j) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                uint32_t d = 0;
                if (FULL || c * (DP / 4) + 32 * j < dim) {
                    w = ld(reinterpret_cast<const uint4 *>(cp) + j);
                    d = ld(reinterpret_cast<const uint32_t *>(sp) + j);
                }
                r.w[i][4 * j] = w.x;
                r.w[i][4 * j + 1] = w.y;
                r.w[i][4 * j + 2] = w.z;
                r.w[i][4 * j + 3] = w.w;
                r.d[i][j] = d;
            }
        }
    }
}

template <int DP, bool FULL>
__device__ __forceinline__ void load_values(const uint8_t *codes, const uint8_t *scales,
                                            const LaneOffsets<DP, FULL> &o, int g, ValueRegs<DP> &r) {
    const int dim = FULL ? DP : o.dim;
    codes += o.vc;
    scales += o.vs;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint8_t *cp = codes + t * 2 * dim;  // four rows on
        const uint8_t *sp = scales + t * (dim / 2);
        r.d[t] = 0;
#pragma unroll
        for (int j = 0; j < ValueRegs<DP>::W; ++j) r.w[t][j] = 0;
        if (FULL || g * (DP / 8) < dim) {
            if constexpr (DP == 64) {
                r.w[t][0] = ld(reinterpret_cast<const uint32_t *>(cp));
                r.d[t] = ld(reinterpret_cast<const uint16_t *>(sp));
            } else if constexpr (DP == 128) {
                const uint2 w = ld(reinterpret_cast<const uint2 *>(cp));
                r.w[t][0] = w.x;
                r.w[t][1] = w.y;
                r.d[t] = ld(reinterpret_cast<const uint16_t *>(sp));
            } else {
                const uint4 w = ld(reinterpret_cast<const uint4 *>(cp));
                r.w[t][0] = w.x;
                r.w[t][1] = w.y;
                r.w[t][2] = w.z;
                r.w[t][3] = w.w;
                r.d[t] = ld(reinterpret_cast<const uint32_t *>(sp));
            }
        }
    }
}

__device__ __forceinline__ uint32_t dup_half(uint32_t d, bool high) { return prmt(d, d, high ? 0x3232u : 0x1010u); }

// Running state of a warp's rows: row 2c + k of each tile of 8.
template <int DP, int NT>
struct AttnState {
    float o[NT][DP / 16][4];
    float off[NT][2], unit[NT][2], l[NT][2];  // RowScale
};

// Groups of a warp's step: 1 and 2 take 102.8 and 96.9 us for 64 sequences of up
// to 8000 tokens (10.0 and 11.6 us for one of 1000).
constexpr int kStepGroups = 2;

// Scores of a group against the rotated queries: s[n] = K q^T.
template <int DP, int NT>
__device__ __forceinline__ void group_scores(const KeyRegs<DP> &r, const uint32_t (&qf)[NT][DP / 16][2],
                                             float (&s)[NT][4], uint32_t lane_base) {
    uint32_t kd[2] = {0u, 0u};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {  // 16 elements: bytes 2i and 2i + 1 of the lane's codes
        if (i % 4 == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) kd[h] = dup_half(r.d[h][i / 8], (i / 4) & 1);
        }
        uint32_t a[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = r.w[h][i / 2];
            a[h] = hmul2((i & 1) ? lut_pair<2>(w, lane_base) : lut_pair<0>(w, lane_base), kd[h]);
            a[2 + h] = hmul2((i & 1) ? lut_pair<3>(w, lane_base) : lut_pair<1>(w, lane_base), kd[h]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(s[n], a[0], a[1], a[2], a[3], qf[n][i][0], qf[n][i][1]);
    }
}

// O^T += V^T P^T of a group.
template <int DP, int NT>
__device__ __forceinline__ void group_values(const ValueRegs<DP> &r, const uint32_t (&pb)[NT][2],
                                             AttnState<DP, NT> &st, uint32_t lane_base) {
#pragma unroll
    for (int half = 0; half < ValueRegs<DP>::H; ++half) {
        const uint32_t d01 = prmt(r.d[0], r.d[1], half ? 0x7632u : 0x5410u);
        const uint32_t d23 = prmt(r.d[2], r.d[3], half ? 0x7632u : 0x5410u);
        constexpr int kWords = ValueRegs<DP>::W / ValueRegs<DP>::H;
#pragma unroll
        for (int jj = 0; jj < kWords; ++jj) {
            const int j = half * kWords + jj;
            // byte b: element 2b (or 2b + 1) of two tokens
            const uint32_t e01 = (r.w[0][j] & 0x0F0F0F0Fu) | ((r.w[1][j] << 4) & 0xF0F0F0F0u);
            const uint32_t f01 = ((r.w[0][j] >> 4) & 0x0F0F0F0Fu) | (r.w[1][j] & 0xF0F0F0F0u);
            const uint32_t e23 = (r.w[2][j] & 0x0F0F0F0Fu) | ((r.w[3][j] << 4) & 0xF0F0F0F0u);
            const uint32_t f23 = ((r.w[2][j] >> 4) & 0x0F0F0F0Fu) | (r.w[3][j] & 0xF0F0F0F0u);
            auto product = [&](auto byte) {
                constexpr int B = decltype(byte)::value;
                const uint32_t a0 = hmul2(lut_pair<B>(e01, lane_base), d01);
                const uint32_t a1 = hmul2(lut_pair<B>(f01, lane_base), d01);
                const uint32_t a2 = hmul2(lut_pair<B>(e23, lane_base), d23);
                const uint32_t a3 = hmul2(lut_pair<B>(f23, lane_base), d23);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(st.o[n][4 * j + B], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            };
            product(std::integral_constant<int, 0>());
            product(std::integral_constant<int, 1>());
            product(std::integral_constant<int, 2>());
            product(std::integral_constant<int, 3>());
        }
    }
}

// Softmax weights of a step's groups under the running maximum, as operands of
// the second product.  TAIL: some tokens are drafted, past the end or without
// a page, and each score is checked; otherwise every token counts.
template <int DP, int NT, bool TAIL>
__device__ __forceinline__ void step_weights(const AttnParams &P, float (&s)[kStepGroups][NT][4],
                                             AttnState<DP, NT> &st, uint32_t (&pb)[kStepGroups][NT][2], int lane,
                                             int token0, int len, const int (&page)[kStepGroups],
                                             const uint64_t (&see)[NT][2]) {
    const int g = lane >> 2;
    const int tok = (g >> 1) + 4 * (g & 1);  // this lane's score rows: tok, tok + 8
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t ok = ~0u;
        if (TAIL) {
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = token0 + q * kGroup + tok + 8 * (i >> 1) - len;
                    const bool sees = page[q] >= 0 && (j < 0 || (j < P.tree && ((see[n][i & 1] >> j) & 1ull)));
                    if (!sees) {
                        ok &= ~(1u << (4 * q + i));
                        s[q][n][i] = kNoMax;
                    }
                }
        }
        float mx[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            mx[k] = kNoMax;
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) mx[k] = fmaxf(mx[k], fmaxf(s[q][n][k], s[q][n][k + 2]));
        }
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(kFull, mx[0], x));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(kFull, mx[1], x));
        }
        if (__any_sync(kFull, outgrown(mx[0], st.unit[n][0], st.off[n][0]) ||
                                  outgrown(mx[1], st.unit[n][1], st.off[n][1]))) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float off = fminf(st.off[n][k], weight_offset(mx[k], st.unit[n][k]));
                const float f = ex2(off - st.off[n][k]);
                st.off[n][k] = off;
                st.l[n][k] *= f;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    st.o[n][i][k] *= f;
                    st.o[n][i][k + 2] *= f;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kStepGroups; ++q) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = ex2(fmaf(s[q][n][i], st.unit[n][i & 1], st.off[n][i & 1]));
                if (TAIL && !((ok >> (4 * q + i)) & 1u)) p[i] = 0.f;
            }
            st.l[n][0] += p[0] + p[2];
            st.l[n][1] += p[1] + p[3];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const __half2 h = __floats2half2_rn(p[2 * k], p[2 * k + 1]);
                pb[q][n][k] = movmatrix(*reinterpret_cast<const uint32_t *>(&h));
            }
        }
    }
}

// Shared memory: prefix sums below the table, which starts at kLutBase and
// ends at kLutBase + 64 KB.
struct AttnShared {
    int prefix[kAttnMaxBatch + 1];
    int scan[32];
};
constexpr int kAttnSmem = (int)(kLutBase + 256 * kLutStep);
constexpr int kMaxSmemBase = 4096;
static_assert(sizeof(AttnShared) + kMaxSmemBase <= kLutBase, "shared memory below the table");

// A value that is the same in every lane, told so.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kFull, x, 0); }

template <int DP, int NT, int WARPS, bool FULL>
__global__ void __launch_bounds__(WARPS * 32, 1) attend_kernel(const AttnParams P) {
    extern __shared__ char smem[];
    AttnShared &sh = *reinterpret_cast<AttnShared *>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const int g = lane >> 2, c = lane & 3;
    fill_lut(tid, WARPS * 32);
    grid_dependency_wait();
    grid_dependents_launch();  // the joining launch may take its place; it waits for this one's end
    scan_sequences(P, sh.prefix, sh.scan, tid, WARPS * 32);
    // defined behind the barrier, so that no lookup is moved in front of it
    uint32_t lane_base;
    asm volatile("mov.u32 %0, %1;" : "=r"(lane_base) : "r"(kLutBase | (uint32_t)(lane * 4)) : "memory");
    const int per_seq = P.c.kv_heads * P.row_tiles;
    const int64_t W = (int64_t)sh.prefix[P.c.batch] * per_seq;
    if (blockIdx.x == 0 && tid == 0) P.header[0] = 0u;  // no wait here that could run out
    // the first warps of all CTAs come first, so that a few ranges spread over the SMs
    const int workers = worker_count(P, W);
    const int me = warp * gridDim.x + blockIdx.x;
    if (me >= workers) return;
    const LaneOffsets<DP, FULL> off(P.c.head_dim, lane);
    int64_t at = quotient(W * me, workers);
    const int64_t end = quotient(W * (me + 1), workers);

    while (at < end) {
        // the unit that holds group `at`
        int lo = 0, hi = P.c.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)sh.prefix[mid] * per_seq <= at) lo = mid;
            else hi = mid - 1;
        }
        const int b = uniform(lo), groups = uniform(sh.prefix[b + 1] - sh.prefix[b]);
        const int64_t in_seq = at - (int64_t)sh.prefix[b] * per_seq;
        const int hr = uniform((int)quotient(in_seq, groups));
        const int head = hr / P.row_tiles, row0 = (hr % P.row_tiles) * NT * 8;
        const int va = uniform((int)(in_seq - (int64_t)hr * groups));
        const int vb = uniform((int)min((int64_t)groups, va + (end - at)));
        at += vb - va;
        const int ga = max(va - P.extra, 0), gb = max(vb - P.extra, 0);
        if (ga >= gb) continue;
        const int len = uniform(min(max(P.lens[b], 0), P.c.pages_per_seq << P.c.page_shift));

        // first loads before the query is rotated
        const int32_t *table = P.c.page_table + b * P.c.table_ld;
        const int shift = P.c.page_shift - 4;  // groups of a page
        const int in_page = (1 << shift) - 1;
        // records of a page, and from a key record to its value record
        const int64_t v_rows = (int64_t)P.c.kv_heads << P.c.page_shift, page_rows = 2 * v_rows;
        const int64_t head_row = (int64_t)head << P.c.page_shift;
        KeyRegs<DP> kr[kStepGroups];
        ValueRegs<DP> vr[kStepGroups];
        // pages and groups are the same for the whole warp, and said to be: the
        // bases below are then computed once per warp
        auto pages_of = [&](int grp, int (&page)[kStepGroups]) {
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) {
                int p = grp + q < gb ? table[(grp + q) >> shift] : -1;
                if (p >= P.c.pages) p = -1;
                page[q] = uniform(p);
            }
        };
        auto record = [&](int page, int grp) { return page * page_rows + head_row + (grp & in_page) * kGroup; };
        auto fetch_keys = [&](const int (&page)[kStepGroups], int grp) {
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) {
                if (page[q] >= 0) {
                    const int64_t rec = record(page[q], grp + q);
                    load_keys<DP, FULL>(P.c.codes + rec * (off.dim / 2),
                                        reinterpret_cast<const uint8_t *>(P.c.scales) + rec * (off.dim / 8), off, c,
                                        kr[q]);
                }
            }
        };
        auto fetch_values = [&](const int (&page)[kStepGroups], int grp) {
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) {
                if (page[q] >= 0) {
                    const int64_t rec = record(page[q], grp + q) + v_rows;
                    load_values<DP, FULL>(P.c.codes + rec * (off.dim / 2),
                                          reinterpret_cast<const uint8_t *>(P.c.scales) + rec * (off.dim / 8), off, g,
                                          vr[q]);
                }
            }
        };
#pragma unroll
        for (int q = 0; q < kStepGroups; ++q) {
            kr[q] = KeyRegs<DP>();
            vr[q] = ValueRegs<DP>();
        }
        const TreeParents tree(P, b, lane);
        int grp = ga;
        int page[kStepGroups], next[kStepGroups];
        pages_of(grp, page);
        pages_of(grp + kStepGroups, next);
        fetch_keys(page, grp);
        fetch_values(page, grp);

        uint32_t qf[NT][DP / 16][2];
        AttnState<DP, NT> st;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = row0 + 8 * n + g;
            const bool valid = row < P.rows;
            const int t = valid ? row / P.group_heads : 0, h = head * P.group_heads + (valid ? row % P.group_heads : 0);
            const int64_t x = b * P.q_batch + t * P.q_token + h * P.q_head;
            float unit;  // of row g's scores
            if (P.qdtype == kF32) unit = rotate_query<kF32, DP>(P, P.q + x * 4, valid, c, qf[n]);
            else if (P.qdtype == kBF16) unit = rotate_query<kBF16, DP>(P, P.q + x * 2, valid, c, qf[n]);
            else unit = rotate_query<kF16, DP>(P, P.q + x * 2, valid, c, qf[n]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                st.unit[n][k] = __shfl_sync(kFull, unit, 4 * (2 * c + k));  // of row 2c + k
                st.off[n][k] = weight_offset(kNoMax, st.unit[n][k]);
                st.l[n][k] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) st.o[n][i][k] = 0.f;
        }

        // keys of the next step load while this step's values are multiplied,
        // its values while the next step's scores are
        while (grp < gb) {
            const int token0 = grp * kGroup;
            bool tail = token0 + kStepGroups * kGroup > len;
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) tail |= page[q] < 0;
            float s[kStepGroups][NT][4];
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) group_scores<DP, NT>(kr[q], qf, s[q], lane_base);
            fetch_keys(next, grp + kStepGroups);
            uint32_t pb[kStepGroups][NT][2];
            if (tail) {
                const TreeWords words(P, tree, lane);
                uint64_t see[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int row = row0 + 8 * n + 2 * c + k;
                        see[n][k] = words.of(min(row / P.group_heads, P.tree - 1));
                    }
                const uint64_t present = words.present();
#pragma unroll
                for (int q = 0; q < kStepGroups; ++q)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        // a record that no query sees counts as zero whatever the memory holds
                        const int j = token0 + q * kGroup + c + 4 * t - len;
                        if (page[q] < 0 || (j >= 0 && (j >= P.tree || !((present >> j) & 1ull)))) vr[q].d[t] = 0;
                    }
                step_weights<DP, NT, true>(P, s, st, pb, lane, token0, len, page, see);
            } else {
                const uint64_t see[NT][2] = {};
                step_weights<DP, NT, false>(P, s, st, pb, lane, token0, len, page, see);
            }
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) group_values<DP, NT>(vr[q], pb[q], st, lane_base);
            grp += kStepGroups;
            fetch_values(next, grp);
#pragma unroll
            for (int q = 0; q < kStepGroups; ++q) page[q] = next[q];
            pages_of(grp + kStepGroups, next);
        }

        // this part of the unit: maxima and sums, and DP / 8 neighbouring
        // elements of two rows for each lane
        const int64_t unit = (int64_t)b * per_seq + hr, slot = unit + me;
        if (lane == 0 && ga == 0) P.span[2 * unit] = me;
        if (lane == 0 && gb == groups - P.extra) P.span[2 * unit + 1] = me;
        uint64_t present = ~0ull;
        if (P.parents) present = TreeWords(P, tree, lane).present();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float l = st.l[n][k];
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l += __shfl_xor_sync(kFull, l, x);
                const int r = 8 * n + 2 * c + k;
                // a token that is not there answers zero
                if (row0 + r < P.rows && !((present >> ((row0 + r) / P.group_heads)) & 1ull)) l = 0.f;
                if (row0 + r < P.rows) {
                    const int64_t at_row = slot * (NT * 8) + r;
                    if (g == 0) reinterpret_cast<float2 *>(P.part_ml)[at_row] = make_float2(-st.off[n][k], l);
                    if (FULL || g * (DP / 8) < P.c.head_dim) {
                        float4 *dst = reinterpret_cast<float4 *>(P.part_o + at_row * off.dim + g * (DP / 8));
#pragma unroll
                        for (int i = 0; i < DP / 16; i += 2)
                            dst[i / 2] = make_float4(st.o[n][i][k], st.o[n][i][k + 2], st.o[n][i + 1][k],
                                                     st.o[n][i + 1][k + 2]);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The parts of each row joined, rotated back, divided and rounded.  CTAs of
// eight warps; a warp takes a row (RW = 1), or all eight share one (RW = 8), as
// they do in any launch where a row has more than kAlone parts (a long sequence
// among short ones: 100000 tokens and 64 times 100, 55 us, with a warp for each
// row 100); a CTA's rows lie far apart, so that such rows seldom meet in one.
// SB: halves of 128 elements.  What bounds this launch is its chain of dependent loads (span, then
// maxima, sums and the first values), so the attention kernel leaves each unit's
// span of slots ready to be read, and values are loaded before their weights are
// known (figures: launch_join_by).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
constexpr int kAlone = 32;

// Reference (log2), sum and values (4 lane + i of each 128) of parts.
template <int SB>
struct JoinState {
    float acc[SB][4], m, l;
};

// Parts [c, end) of the slots from s0, row r of each; up to 32 at a time: a lane
// takes one part's maximum and sum, then all lanes its values.
template <int AHEAD, int SB>
__device__ __forceinline__ void join_parts(const AttnParams &P, int64_t s0, int r, int c, int end, int lane,
                                           JoinState<SB> &st) {
    const int D = P.c.head_dim;
    st = JoinState<SB>{};
    st.m = kNoMax;
    for (; c < end; c += 32) {
        float2 p = make_float2(kNoMax, 0.f);
        if (c + lane < end) p = reinterpret_cast<const float2 *>(P.part_ml)[(s0 + c + lane) * P.tile_rows + r];
        const int count = min(32, end - c);
        const float *src = P.part_o + ((s0 + c) * P.tile_rows + r) * D + 4 * lane;
        float4 v[AHEAD][SB];
        auto values = [&](int j, float4 (&o)[SB]) {
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                o[sb] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < count && sb * 128 + 4 * lane < D)
                    o[sb] = *reinterpret_cast<const float4 *>(src + (int64_t)j * P.tile_rows * D + sb * 128);
            }
        };
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) values(j, v[j]);
        float mx = fmaxf(st.m, p.y != 0.f ? p.x : kNoMax);  // (a NaN sum counts: it has to reach the output)
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, x));
        const float f = p.y != 0.f ? ex2(p.x - mx) : 0.f;
        float sum = f * p.y;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(kFull, sum, x);
        const float old = ex2(st.m - mx);
        st.l = st.l * old + sum;
        st.m = mx;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.acc[sb][i] *= old;
        for (int j = 0; j < count; j += AHEAD) {
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const float fj = j + q < count ? __shfl_sync(kFull, f, j + q) : 0.f;
                // (a part without a token may never have been written: its values do not count)
                if (fj != 0.f) {
#pragma unroll
                    for (int sb = 0; sb < SB; ++sb) {
                        st.acc[sb][0] += fj * v[q][sb].x;
                        st.acc[sb][1] += fj * v[q][sb].y;
                        st.acc[sb][2] += fj * v[q][sb].z;
                        st.acc[sb][3] += fj * v[q][sb].w;
                    }
                }
                values(j + AHEAD + q, v[q]);
            }
        }
    }
}

template <int OT, int RW, int SB>
__global__ void __launch_bounds__(kJoinWarps * 32, RW == 1 ? 4 : 2) join_kernel(const AttnParams P) {
    constexpr int kRows = kJoinWarps / RW;  // of a CTA
    // parts whose values are on their way: many in a launch of few rows; of many
    // rows, as many as leave the registers for other warps (4 instead of 2: 182
    // against 173 us for 131072 rows; 4 instead of 8: 17.6 against 16.5 us for 32)
    constexpr int kAhead = RW == 1 ? 2 : 8;
    __shared__ float so[kJoinWarps][128 * SB];
    __shared__ float sl[kJoinWarps], sm[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = P.c.batch * P.c.kv_heads * P.rows, grid = (int)gridDim.x;
    const int index = warp / RW * grid + (int)blockIdx.x;
    const int bh = index / P.rows, row = index % P.rows;
    const int b = bh / P.c.kv_heads, head = bh % P.c.kv_heads;
    const int t = row / P.group_heads, h = head * P.group_heads + row % P.group_heads;
    const int D = P.c.head_dim;
    uint32_t flips[SB];
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) flips[sb] = c_sign_words.w[sb * 4 + lane / 8] >> (4 * (lane & 7));
    // lane k: row k of the CTA, its place in its tile, its unit
    const int of_lane = min(lane, kRows - 1) * grid + (int)blockIdx.x;
    const int lane_row = of_lane % P.rows;
    const int lane_r = lane_row % P.tile_rows;
    const int64_t unit = (int64_t)(of_lane / P.rows) * P.row_tiles + lane_row / P.tile_rows;
    grid_dependency_wait();
    grid_dependents_launch();
    int64_t slot = 0;
    int parts = 0;
    if (of_lane < rows) {
        // its workers; a call that gave up left some of these unwritten, so they are bounded
        const int2 span = *reinterpret_cast<const int2 *>(P.span + 2 * unit);
        const int first = min(max(span.x, 0), P.workers - 1);
        const int last = min(max(span.y, first), P.workers - 1);
        slot = (unit + first) * P.parts;       // the unit's first slot
        parts = (last - first + 1) * P.parts;  // and how many
    }
    auto finish = [&](JoinState<SB> &st) {
        const float inv = st.l != 0.f ? 0.03125f / st.l : 0.f;  // no token: zeros
        char *out = P.out + (b * P.o_batch + t * P.o_token + h * P.o_head) * ElemSize<OT>::value;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            if (sb * 128 >= D) break;
            const int e = sb * 128 + 4 * lane;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = st.acc[sb][i] * inv;
            fwht32_warp(v, lane & 7);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = flip(v[i], (flips[sb] << (31 - i)) & 0x80000000u);
            if (e < D) store4<OT>(out + (int64_t)e * ElemSize<OT>::value, v);
        }
    };
    if (RW == 1) {
        const int n = __shfl_sync(kFull, parts, warp);
        if (n > 0 && n <= kAlone) {
            JoinState<SB> st;
            join_parts<kAhead, SB>(P, __shfl_sync(kFull, slot, warp), __shfl_sync(kFull, lane_r, warp), 0, n, lane, st);
            finish(st);
        }
    }
    // rows that all warps share (every warp knows them)
    uint32_t shared = __ballot_sync(kFull, lane < kRows && parts > (RW == 1 ? kAlone : 0));
#pragma unroll 1
    for (; shared; shared &= shared - 1) {
        const int k = __ffs(shared) - 1, n = __shfl_sync(kFull, parts, k);
        JoinState<SB> st;
        join_parts<kAhead, SB>(P, __shfl_sync(kFull, slot, k), __shfl_sync(kFull, lane_r, k), n * warp / kJoinWarps,
                               n * (warp + 1) / kJoinWarps, lane, st);
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
            *reinterpret_cast<float4 *>(&so[warp][sb * 128 + 4 * lane]) =
                make_float4(st.acc[sb][0], st.acc[sb][1], st.acc[sb][2], st.acc[sb][3]);
        if (lane == 0) {
            sl[warp] = st.l;
            sm[warp] = st.m;
        }
        __syncthreads();
        if (warp == k * RW) {
            float mx = kNoMax;
#pragma unroll
            for (int x = 0; x < kJoinWarps; ++x) mx = fmaxf(mx, sm[x]);
            st = JoinState<SB>{};
#pragma unroll
            for (int x = 0; x < kJoinWarps; ++x) {
                const float f = ex2(sm[x] - mx);
                st.l += f * sl[x];
#pragma unroll
                for (int sb = 0; sb < SB; ++sb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st.acc[sb][i] += f * so[x][sb * 128 + 4 * lane + i];
            }
            finish(st);
        }
        if (RW == 1) __syncthreads();
    }
    // what the CTAs reported, into the header (behind the rows: an extra CTA, told apart
    // at the start, cost launches without a status 0.2 of 14.6 us)
    if (P.status && blockIdx.x == gridDim.x - 1 && warp == kJoinWarps - 1) {
        unsigned word = 0;
        for (int i = lane; i < P.workers; i += 32) word |= P.status[i];
        word = __reduce_or_sync(kFull, word);
        if (lane == 0) P.header[0] = word;
    }
}

// Which kernel runs, and how it cuts the work.
struct AttnPlan {
    bool tc;  // the tcgen05 kernel
    int dp, nt, warps;
    int rows, row_tiles, tile_rows, group, workers, least, extra, parts;
    int64_t slots;
};

AttnPlan plan_attention(int64_t batch, int tree, int heads, int kv_heads, int head_dim, int sm_count) {
    AttnPlan p = {};
    p.rows = tree * (heads / kv_heads);
    p.tc = p.rows > kTcLeastRows && tc_attention_fits(head_dim);
    if (p.tc) {
        p.tile_rows = tc_attention_tile_rows(p.rows);
        p.parts = p.tile_rows == 128 ? 2 : 1;
        p.group = 128;
        p.workers = sm_count;
        p.least = 1;
        p.extra = kTcExtra;
    } else {
        // tiles of 8 rows, or 16 where a (sequence, head) has more than 8 rows
        // and the accumulators of 16 fit the registers (head dimension up to
        // 128): 16 rows over 64 sequences of 4000 tokens as one tile 127 us, as
        // two 169.  16 warps where 128 registers hold a tile: 8 rows over the
        // same 92 us, with 8 warps 106 (one sequence of 30000 tokens, whose
        // parts have to be joined, 28 and 24)
        p.dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
        p.nt = p.rows > 8 && p.dp <= 128 ? 2 : 1;
        p.warps = p.nt == 2 || p.dp == 256 ? 8 : 16;
        p.tile_rows = 8 * p.nt;
        p.parts = 1;
        p.group = kGroup;
        p.workers = sm_count * p.warps;
        p.least = kLeastGroups;
        p.extra = kExtraGroups;
    }
    p.row_tiles = (p.rows + p.tile_rows - 1) / p.tile_rows;
    p.slots = (batch * kv_heads * p.row_tiles + p.workers) * p.parts;
    return p;
}

template <int DP, int NT, int WARPS, bool FULL>
cudaError_t launch_attend_as(const AttnParams &P, cudaStream_t stream) {
    // the table stands at a fixed address: dynamic shared memory has to begin
    // low enough for what lies below it
    int dev = 0, reserved = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
    if (e == cudaSuccess && reserved > kMaxSmemBase) e = cudaErrorInvalidValue;
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attend_kernel<DP, NT, WARPS, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kAttnSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(attend_kernel<DP, NT, WARPS, FULL>, P.workers / WARPS, WARPS * 32, kAttnSmem, stream, P);
}

template <int DP, int NT, int WARPS>
cudaError_t launch_attend(const AttnParams &P, cudaStream_t stream) {
    return P.c.head_dim == DP ? launch_attend_as<DP, NT, WARPS, true>(P, stream)
                              : launch_attend_as<DP, NT, WARPS, false>(P, stream);
}

template <int OT, int RW>
cudaError_t launch_join_as(const AttnParams &P, cudaStream_t stream) {
    const int64_t warps = (int64_t)P.c.batch * P.c.kv_heads * P.rows * RW;
    const unsigned grid = (unsigned)((warps + kJoinWarps - 1) / kJoinWarps);
    return P.c.head_dim <= 128 ? launch_dependent(join_kernel<OT, RW, 1>, grid, kJoinWarps * 32, 0, stream, P)
                               : launch_dependent(join_kernel<OT, RW, 2>, grid, kJoinWarps * 32, 0, stream, P);
}

// Eight warps share a row where rows are few and their parts (about workers /
// units + 1) many; else a warp takes a row.  Whole call, eight warps against
// one: 32 rows of up to 297 parts 16.5 and 75 us; 256 rows of 38 parts 33 and 48;
// 1024 rows of 10 parts 23.5 and 18.5; 2048 rows of 10 parts 46.5 and 35.
constexpr int64_t kManyParts = 16;
constexpr int64_t kFewRows = 148 * 8;

template <int OT>
cudaError_t launch_join_by(const AttnParams &P, cudaStream_t stream) {
    const int64_t pairs = (int64_t)P.c.batch * P.c.kv_heads;
    const int64_t parts = (int64_t)P.workers * P.parts / (pairs * P.row_tiles) + 1;
    return parts > kManyParts && pairs * P.rows <= kFewRows ? launch_join_as<OT, 8>(P, stream)
                                                            : launch_join_as<OT, 1>(P, stream);
}

}  // namespace

cudaError_t launch_join(const AttnParams &P, int odtype, cudaStream_t stream) {
    if (odtype == kF32) return launch_join_by<kF32>(P, stream);
    return odtype == kBF16 ? launch_join_by<kBF16>(P, stream) : launch_join_by<kF16>(P, stream);
}

// Workspace: a 256-byte header (status word), the CTAs' status words, the units'
// spans, the parts' references and sums, their values.
size_t attention_workspace_bytes(int64_t batch, int tree, int heads, int kv_heads, int head_dim, int sm_count) {
    const AttnPlan p = plan_attention(batch, tree, heads, kv_heads, head_dim, sm_count);
    return 256 + round_up((size_t)p.workers * 4, 256) + round_up((size_t)batch * kv_heads * p.row_tiles * 8, 256) +
           round_up((size_t)p.slots * p.tile_rows * 8, 256) + (size_t)p.slots * p.tile_rows * head_dim * 4;
}

cudaError_t launch_attention(const AttentionJob &j, int sm_count, cudaStream_t stream) {
    const AttnPlan plan = plan_attention(j.c.batch, j.tree, j.heads, j.c.kv_heads, j.c.head_dim, sm_count);
    AttnParams P;
    P.c = j.c;
    P.lens = j.lens;
    P.parents = j.parents;
    P.parents_ld = j.parents_ld;
    P.q = static_cast<const char *>(j.q);
    P.q_batch = j.q_batch;
    P.q_token = j.q_token;
    P.q_head = j.q_head;
    P.out = static_cast<char *>(j.out);
    P.o_batch = j.o_batch;
    P.o_token = j.o_token;
    P.o_head = j.o_head;
    P.tree = j.tree;
    P.heads = j.heads;
    P.group_heads = j.heads / j.c.kv_heads;
    P.rows = plan.rows;
    P.row_tiles = plan.row_tiles;
    P.qdtype = j.qdtype;
    P.q_factor = j.scale * (1.44269504088896340736f * 0.03125f);
    P.group = plan.group;
    P.workers = plan.workers;
    P.least = plan.least;
    P.extra = plan.extra;
    P.parts = plan.parts;
    P.tile_rows = plan.tile_rows;
    P.header = reinterpret_cast<unsigned *>(j.workspace);
    P.inject_skip = (debug_flags() & kDebugSkipCacheKeys) ? 1 : 0;
    P.timeout_cycles = P.inject_skip ? 10000000ll : 2000000000ll;  // about 5 ms, a second
    P.inject_tmem = (debug_flags() & kDebugNoTensorMemory) ? 1 : 0;
    char *ws = j.workspace + 256;
    P.status = plan.tc ? reinterpret_cast<unsigned *>(ws) : nullptr;
    ws += round_up((size_t)plan.workers * 4, 256);
    P.span = reinterpret_cast<int *>(ws);
    ws += round_up((size_t)j.c.batch * j.c.kv_heads * plan.row_tiles * 8, 256);
    P.part_ml = reinterpret_cast<float *>(ws);
    ws += round_up((size_t)plan.slots * plan.tile_rows * 8, 256);
    P.part_o = reinterpret_cast<float *>(ws);

    cudaError_t e;
    if (plan.tc) e = launch_tc_attention(P, stream);
    else if (plan.dp == 64) e = plan.nt == 1 ? launch_attend<64, 1, 16>(P, stream) : launch_attend<64, 2, 8>(P, stream);
    else if (plan.dp == 128)
        e = plan.nt == 1 ? launch_attend<128, 1, 16>(P, stream) : launch_attend<128, 2, 8>(P, stream);
    else e = launch_attend<256, 1, 8>(P, stream);
    return e != cudaSuccess ? e : launch_join(P, j.odtype, stream);
}

}  // namespace tq
