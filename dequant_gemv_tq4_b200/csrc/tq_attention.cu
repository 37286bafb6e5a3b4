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
// attend_kernel (mma.sync, tiles of 8 or 16 rows).  One CTA per SM; every
// warp takes groups of 16 tokens on its own:
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
// query (as in the products of this library), and the softmax weights, which
// are scaled by 2^14 so that weights down to 2^-38 of the largest survive.
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kGroup = 16;               // tokens of a group
constexpr uint32_t kLutBase = 0x10000u;  // shared-memory address of the centroid table
constexpr uint32_t kLutStep = 256;       // bytes between its rows (128 used)
constexpr float kWeightExp = 14.0f;      // softmax weights are held times 2^14
constexpr int kSmemLimit = 227 * 1024;

struct AttnParams {
    KvCache c;
    const int32_t *lens, *parents;  // parents null: a chain
    int64_t parents_ld;
    const char *q;
    int64_t q_batch, q_token, q_head;  // elements
    char *out;
    int64_t o_batch, o_token, o_head;
    int tree, heads, group_heads;  // query heads per key/value head
    int rows, row_tiles;           // rows of a (sequence, head), tiles of them
    int qdtype;
    float scale_log2;
    int *prefix;     // [batch + 1] groups before each sequence
    float *part_ml;  // [slots][rows of a tile][2]: maximum, sum
    float *part_o;   // [slots][rows of a tile][head_dim]
    int grid;
};

// Tokens that sequence b attends over, drafted ones included, within its table.
__device__ __forceinline__ int seq_tokens(const AttnParams &P, int len) {
    const int64_t cap = (int64_t)P.c.pages_per_seq << P.c.page_shift;
    const int64_t n = (int64_t)max(len, 0) + P.tree;
    return (int)(n < cap ? n : cap);
}

// The split of W groups over the CTAs: CTA i takes [i W / g, (i + 1) W / g)
// with g CTAs at work, at least `least` groups each.
__device__ __forceinline__ int cta_count(int64_t W, int grid, int least) {
    const int64_t g = (W + least - 1) / least;
    return (int)(g < grid ? (g < 1 ? 1 : g) : grid);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

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

// Which drafted tokens each drafted token sees: itself and its ancestors, a
// 64-bit word per token, 0 for a token that is not there (a parent that is
// neither -1 nor an earlier token, its own or an ancestor's).  One warp, six
// rounds of pointer doubling; `ptr` is scratch for 64 ints.
__device__ __forceinline__ void ancestor_words(const AttnParams &P, int b, uint64_t *word, int *ptr, int lane) {
#pragma unroll
    for (int i = lane; i < kAttnMaxTree; i += 32) {
        int par = i - 1;
        if (i >= P.tree) par = -2;
        else if (P.parents) par = P.parents[b * P.parents_ld + i];
        ptr[i] = par < -1 || par >= i ? -2 : par;
        word[i] = 1ull << i;
    }
    __syncwarp();
    for (int hop = 1; hop < kAttnMaxTree; hop <<= 1) {
        uint64_t w[2];
        int p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = lane + 32 * k;
            w[k] = word[i];
            p[k] = ptr[i];
            if (p[k] >= 0) {
                w[k] |= word[p[k]];
                p[k] = ptr[p[k]];
            }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            word[lane + 32 * k] = w[k];
            ptr[lane + 32 * k] = p[k];
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = lane; i < kAttnMaxTree; i += 32)
        if (ptr[i] == -2) word[i] = 0;
    __syncwarp();
}

// One row's rotated query, fp16, into dst[0 .. DP): lane l holds elements
// 4l .. 4l+3 of each 128; columns past the head dimension and rows past the
// tile are zero.
template <int DT, int DP>
__device__ __forceinline__ void rotate_query(const AttnParams &P, const char *x, bool valid, uint32_t *dst, int lane) {
#pragma unroll
    for (int sb = 0; sb < (DP + 127) / 128; ++sb) {
        const int e = sb * 128 + 4 * lane;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (valid && e < P.c.head_dim) load4<DT>(x + (int64_t)e * ElemSize<DT>::value, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = flip(v[i], sign_mask(e + i));
        fwht32_warp(v, lane & 7);
        __half2 a = __floats2half2_rn(v[0] * 0.03125f, v[1] * 0.03125f);
        __half2 c = __floats2half2_rn(v[2] * 0.03125f, v[3] * 0.03125f);
        if (e < DP)
            *reinterpret_cast<uint2 *>(dst + e / 2) =
                make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&c));
    }
}

// What a lane holds of one group of 16 tokens.
template <int DP>
struct GroupRegs {
    static constexpr int KW = DP / 32;  // code words of a key row (DP / 4 elements)
    static constexpr int KD = DP / 64;  // its half-block scales
    static constexpr int VW = DP / 64;  // code words of a value row (DP / 8 elements)
    static constexpr int VD = DP < 256 ? 1 : 2;
    uint32_t k[2][KW];
    uint32_t kd[2][(KD + 1) / 2];
    uint32_t v[4][VW];
    uint32_t vd[4];
};

// Key rows of a lane (l = 4 g + c): tokens 4 (g / 2) + g % 2 and that + 2,
// elements DP/4 * c ...; value rows: tokens 4 c .. 4 c + 3, elements DP/8 * g ...
// This is the order in which S^T's accumulator, transposed by movmatrix, is
// the weights operand of the second product.
template <int DP>
__device__ __forceinline__ void load_group(const AttnParams &P, int64_t page, int head, int row0, int lane,
                                           GroupRegs<DP> &r) {
    using R = GroupRegs<DP>;
    const int g = lane >> 2, c = lane & 3, D = P.c.head_dim;
    const int64_t krec = ((page * 2 * P.c.kv_heads + head) << P.c.page_shift) + row0;
    const int64_t vrec = krec + ((int64_t)P.c.kv_heads << P.c.page_shift);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t rec = krec + 4 * (g >> 1) + (g & 1) + 2 * i;
        const uint8_t *codes = P.c.codes + rec * (D / 2) + c * (DP / 8);
        const uint16_t *scales = P.c.scales + rec * (D / 16) + c * R::KD;
        if constexpr (DP == 64) {
            uint2 w = make_uint2(0u, 0u);
            r.kd[i][0] = 0;
            if (16 * c < D) {
                w = __ldg(reinterpret_cast<const uint2 *>(codes));
                r.kd[i][0] = __ldg(scales);
            }
            r.k[i][0] = w.x;
            r.k[i][1] = w.y;
        } else {
#pragma unroll
            for (int j = 0; j < DP / 128; ++j) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                uint32_t d = 0;
                if (c * (DP / 4) + 32 * j < D) {
                    w = __ldg(reinterpret_cast<const uint4 *>(codes) + j);
                    d = __ldg(reinterpret_cast<const uint32_t *>(scales) + j);
                }
                r.k[i][4 * j] = w.x;
                r.k[i][4 * j + 1] = w.y;
                r.k[i][4 * j + 2] = w.z;
                r.k[i][4 * j + 3] = w.w;
                r.kd[i][j] = d;
            }
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t rec = vrec + 4 * c + t;
        const uint8_t *codes = P.c.codes + rec * (D / 2) + g * (DP / 16);
        const uint16_t *scales = P.c.scales + rec * (D / 16) + (g * (DP / 8)) / 16;
        r.vd[t] = 0;
#pragma unroll
        for (int j = 0; j < R::VW; ++j) r.v[t][j] = 0;
        if (g * (DP / 8) < D) {
            if constexpr (DP == 64) {
                r.v[t][0] = __ldg(reinterpret_cast<const uint32_t *>(codes));
                r.vd[t] = __ldg(scales);
            } else if constexpr (DP == 128) {
                const uint2 w = __ldg(reinterpret_cast<const uint2 *>(codes));
                r.v[t][0] = w.x;
                r.v[t][1] = w.y;
                r.vd[t] = __ldg(scales);
            } else {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(codes));
                r.v[t][0] = w.x;
                r.v[t][1] = w.y;
                r.v[t][2] = w.z;
                r.v[t][3] = w.w;
                r.vd[t] = __ldg(reinterpret_cast<const uint32_t *>(scales));
            }
        }
    }
}

__device__ __forceinline__ uint32_t dup_half(uint32_t d, bool high) { return prmt(d, d, high ? 0x3232u : 0x1010u); }

template <int DP, int NT>
struct AttnState {
    float o[NT][DP / 16][4];
    float m[NT][2], l[NT][2];
};

// One group: scores, mask, running softmax, weighted values.  `tail`: some of
// its tokens are drafted, past the end, or without a page.
template <int DP, int NT>
__device__ __forceinline__ void attend_group(const AttnParams &P, const GroupRegs<DP> &r, const uint32_t (&qf)[NT][DP / 16][2],
                                             AttnState<DP, NT> &st, uint32_t lane_base, int lane, bool tail,
                                             bool has_page, int token0, int len, const uint64_t (&see)[NT][2],
                                             const uint64_t *word) {
    const int g = lane >> 2, c = lane & 3;
    float s[NT][2][4];  // two accumulators, for shorter chains of products
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][0][i] = s[n][1][i] = 0.f;
    uint32_t kd[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {  // 16 elements: bytes 2i and 2i + 1 of the lane's codes
        if (i % 4 == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) kd[h] = dup_half(r.kd[h][i / 8], (i / 4) & 1);
        }
        uint32_t a[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = r.k[h][i / 2];
            a[h] = hmul2((i & 1) ? lut_pair<2>(w, lane_base) : lut_pair<0>(w, lane_base), kd[h]);
            a[2 + h] = hmul2((i & 1) ? lut_pair<3>(w, lane_base) : lut_pair<1>(w, lane_base), kd[h]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(s[n][i & 1], a[0], a[1], a[2], a[3], qf[n][i][0], qf[n][i][1]);
    }

    const int tok = 4 * (g >> 1) + (g & 1);  // this lane's score rows: tok, tok + 2
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = (s[n][0][i] + s[n][1][i]) * P.scale_log2;
        if (tail) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = token0 + tok + 2 * (i >> 1) - len;
                const bool ok = has_page && (j < 0 || (j < P.tree && ((see[n][i & 1] >> j) & 1ull)));
                if (!ok) x[i] = -INFINITY;
            }
        }
        float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
        for (int k = 4; k <= 16; k <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(kFull, mx[0], k));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(kFull, mx[1], k));
        }
        const bool grows = mx[0] > st.m[n][0] || mx[1] > st.m[n][1];
        if (__any_sync(kFull, grows)) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float nm = fmaxf(st.m[n][k], mx[k]);
                // rows without any token so far have nothing to rescale
                const float f = st.m[n][k] == -INFINITY ? 0.f : ex2(st.m[n][k] - nm);
                st.m[n][k] = nm;
                st.l[n][k] *= f;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    st.o[n][i][k] *= f;
                    st.o[n][i][k + 2] *= f;
                }
            }
        }
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float m = st.m[n][i & 1];
            p[i] = m == -INFINITY ? 0.f : ex2(x[i] - (m - kWeightExp));
        }
        st.l[n][0] += p[0] + p[2];
        st.l[n][1] += p[1] + p[3];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const __half2 h = __floats2half2_rn(p[2 * k], p[2 * k + 1]);
            pb[n][k] = movmatrix(*reinterpret_cast<const uint32_t *>(&h));
        }
    }

    // scales of the lane's four value rows; a row that no query sees counts as
    // zero whatever the memory holds
    uint32_t vd[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        vd[t] = r.vd[t];
        if (tail) {
            const int j = token0 + 4 * c + t - len;
            const bool there = has_page && (j < 0 || (j < P.tree && word[j] != 0));
            if (!there) vd[t] = 0;
        }
    }
#pragma unroll
    for (int half = 0; half < GroupRegs<DP>::VD; ++half) {
        const uint32_t d01 = prmt(vd[0], vd[1], half ? 0x7632u : 0x5410u);
        const uint32_t d23 = prmt(vd[2], vd[3], half ? 0x7632u : 0x5410u);
        constexpr int kWords = GroupRegs<DP>::VW / GroupRegs<DP>::VD;
#pragma unroll
        for (int jj = 0; jj < kWords; ++jj) {
            const int j = half * kWords + jj;
            // byte b: element 2b (or 2b + 1) of two tokens
            const uint32_t e01 = (r.v[0][j] & 0x0F0F0F0Fu) | ((r.v[1][j] << 4) & 0xF0F0F0F0u);
            const uint32_t f01 = ((r.v[0][j] >> 4) & 0x0F0F0F0Fu) | (r.v[1][j] & 0xF0F0F0F0u);
            const uint32_t e23 = (r.v[2][j] & 0x0F0F0F0Fu) | ((r.v[3][j] << 4) & 0xF0F0F0F0u);
            const uint32_t f23 = ((r.v[2][j] >> 4) & 0x0F0F0F0Fu) | (r.v[3][j] & 0xF0F0F0F0u);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t a[4];
                if (b == 0) {
                    a[0] = lut_pair<0>(e01, lane_base); a[1] = lut_pair<0>(f01, lane_base);
                    a[2] = lut_pair<0>(e23, lane_base); a[3] = lut_pair<0>(f23, lane_base);
                } else if (b == 1) {
                    a[0] = lut_pair<1>(e01, lane_base); a[1] = lut_pair<1>(f01, lane_base);
                    a[2] = lut_pair<1>(e23, lane_base); a[3] = lut_pair<1>(f23, lane_base);
                } else if (b == 2) {
                    a[0] = lut_pair<2>(e01, lane_base); a[1] = lut_pair<2>(f01, lane_base);
                    a[2] = lut_pair<2>(e23, lane_base); a[3] = lut_pair<2>(f23, lane_base);
                } else {
                    a[0] = lut_pair<3>(e01, lane_base); a[1] = lut_pair<3>(f01, lane_base);
                    a[2] = lut_pair<3>(e23, lane_base); a[3] = lut_pair<3>(f23, lane_base);
                }
                a[0] = hmul2(a[0], d01);
                a[1] = hmul2(a[1], d01);
                a[2] = hmul2(a[2], d23);
                a[3] = hmul2(a[3], d23);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816(st.o[n][4 * j + b], a[0], a[1], a[2], a[3], pb[n][0], pb[n][1]);
            }
        }
    }
}

// Shared memory below the table: prefix sums, ancestor words, the rotated
// queries, the warps' maxima and sums; above it the warps' partial results.
constexpr uint32_t kLowBytes = 60 * 1024;

template <int DP, int NT>
struct AttnShared {
    static constexpr int kRowWords = DP / 2 + 4;  // a query row, padded against bank conflicts
    int prefix[kAttnMaxBatch + 1];
    int scan[32];
    uint64_t word[kAttnMaxTree];
    int ptr[kAttnMaxTree];
    uint32_t q[NT * 8 * kRowWords];
    float m[16][NT * 8], l[16][NT * 8];
};

template <int DP, int NT, int WARPS>
constexpr int attn_smem() {
    return (int)(kLutBase + 256 * kLutStep) + WARPS * 8 * (DP + 4) * 4;
}

// Exclusive prefix of the sequences' groups into `prefix`, by the whole CTA.
__device__ __forceinline__ void scan_sequences(const AttnParams &P, int *prefix, int *scan, int tid, int threads) {
    const int per = (P.c.batch + threads - 1) / threads;
    int sum = 0;
    for (int i = tid * per; i < min(P.c.batch, (tid + 1) * per); ++i)
        sum += (seq_tokens(P, P.lens[i]) + kGroup - 1) / kGroup;
    int inc = sum;
    const int lane = tid & 31;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(kFull, inc, k);
        if (lane >= k) inc += o;
    }
    if (lane == 31) scan[tid >> 5] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < (tid >> 5); ++w) base += scan[w];
    int at = base + inc - sum;
    for (int i = tid * per; i < min(P.c.batch, (tid + 1) * per); ++i) {
        prefix[i] = at;
        at += (seq_tokens(P, P.lens[i]) + kGroup - 1) / kGroup;
    }
    if (tid == threads - 1) prefix[P.c.batch] = base + inc;
    __syncthreads();
}

template <int DP, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) attend_kernel(const AttnParams P) {
    using S = AttnShared<DP, NT>;
    static_assert(sizeof(S) <= kLowBytes, "shared memory below the table");
    extern __shared__ char smem[];
    S &sh = *reinterpret_cast<S *>(smem);
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    float *red = reinterpret_cast<float *>(smem + (kLutBase + 256 * kLutStep - base));
    constexpr int kRedRow = DP + 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    grid_dependents_launch();  // the joining launch may take its place; it waits for this one's end

    fill_lut(tid, WARPS * 32);
    scan_sequences(P, sh.prefix, sh.scan, tid, WARPS * 32);
    // defined behind the barrier, so that no lookup is moved in front of it
    uint32_t lane_base;
    asm volatile("mov.u32 %0, %1;" : "=r"(lane_base) : "r"(kLutBase | (uint32_t)(lane * 4)) : "memory");
    const int per_seq = P.c.kv_heads * P.row_tiles;
    const int64_t W = (int64_t)sh.prefix[P.c.batch] * per_seq;
    if (blockIdx.x == 0)
        for (int i = tid; i <= P.c.batch; i += WARPS * 32) P.prefix[i] = sh.prefix[i];
    const int ctas = cta_count(W, P.grid, WARPS);
    if (blockIdx.x >= ctas) return;
    int64_t at = W * blockIdx.x / ctas;
    const int64_t end = W * (blockIdx.x + 1) / ctas;

    while (at < end) {
        // the unit that holds group `at`
        int lo = 0, hi = P.c.batch - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)sh.prefix[mid] * per_seq <= at) lo = mid;
            else hi = mid - 1;
        }
        const int b = lo, groups = sh.prefix[b + 1] - sh.prefix[b];
        const int64_t in_seq = at - (int64_t)sh.prefix[b] * per_seq;
        const int hr = (int)(in_seq / groups);
        const int head = hr / P.row_tiles, row0 = (hr % P.row_tiles) * NT * 8;
        const int ga = (int)(in_seq - (int64_t)hr * groups);
        const int gb = (int)min((int64_t)groups, ga + (end - at));
        const int len = min(max(P.lens[b], 0), (int)min((int64_t)INT32_MAX, (int64_t)P.c.pages_per_seq << P.c.page_shift));

        // first loads before the query is rotated
        const int32_t *table = P.c.page_table + b * P.c.table_ld;
        const int shift = P.c.page_shift - 4;  // groups of a page
        const int in_page = (1 << shift) - 1;
        GroupRegs<DP> next;
        bool next_page = false;
        auto fetch = [&](int grp) {
            const int64_t page = table[grp >> shift];
            next_page = page >= 0 && page < P.c.pages;
            if (next_page) load_group<DP>(P, page, head, (grp & in_page) * kGroup, lane, next);
            else next = GroupRegs<DP>();
        };
        int grp = ga + warp;
        if (grp < gb) fetch(grp);

        if (warp == WARPS - 1) ancestor_words(P, b, sh.word, sh.ptr, lane);
        for (int r = warp; r < NT * 8; r += WARPS) {
            const int row = row0 + r;
            const int t = row / P.group_heads, h = head * P.group_heads + row % P.group_heads;
            const bool valid = row < P.rows;
            const int64_t off = b * P.q_batch + t * P.q_token + h * P.q_head;
            uint32_t *dst = sh.q + r * S::kRowWords;
            if (P.qdtype == kF32) rotate_query<kF32, DP>(P, P.q + off * 4, valid, dst, lane);
            else if (P.qdtype == kBF16) rotate_query<kBF16, DP>(P, P.q + off * 2, valid, dst, lane);
            else rotate_query<kF16, DP>(P, P.q + off * 2, valid, dst, lane);
        }
        __syncthreads();

        // query fragments: row g of each tile of 8, this lane's DP / 4 elements
        uint32_t qf[NT][DP / 16][2];
        uint64_t see[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t *src = sh.q + (8 * n + g) * S::kRowWords + c * (DP / 8);
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src + 2 * i);
                qf[n][i][0] = w.x;
                qf[n][i][1] = w.y;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = row0 + 8 * n + 2 * c + k;
                see[n][k] = row < P.rows ? sh.word[row / P.group_heads] : 0;
            }
        }
        AttnState<DP, NT> st;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                st.m[n][k] = -INFINITY;
                st.l[n][k] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) st.o[n][i][k] = 0.f;
        }
        while (grp < gb) {
            const GroupRegs<DP> cur = next;
            const bool has_page = next_page;
            const int token0 = grp * kGroup;
            grp += WARPS;
            if (grp < gb) fetch(grp);
            const bool tail = token0 + kGroup > len || !has_page;
            attend_group<DP, NT>(P, cur, qf, st, lane_base, lane, tail, has_page, token0, len, see, sh.word);
        }

        // the warps' parts joined: maxima and sums first, then the values
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float l = st.l[n][k];
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l += __shfl_xor_sync(kFull, l, x);
                if (g == 0) {
                    sh.m[warp][8 * n + 2 * c + k] = st.m[n][k];
                    sh.l[warp][8 * n + 2 * c + k] = l;
                }
            }
        }
        __syncthreads();
        const int64_t unit = (int64_t)b * per_seq + hr;
        const int64_t slot = unit + blockIdx.x;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 8 * n + 2 * c + k;
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sh.m[w][r]);
                const float f = st.m[n][k] == -INFINITY ? 0.f : ex2(st.m[n][k] - mx);
                float *dst = red + (warp * 8 + 2 * c + k) * kRedRow + 2 * g;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i)  // elements DP/8 g + 2 i and + 1 at 16 i + 2 g
                    *reinterpret_cast<float2 *>(dst + 16 * i) = make_float2(st.o[n][i][k] * f, st.o[n][i][k + 2] * f);
            }
            __syncthreads();
            for (int i = tid; i < 8 * DP; i += WARPS * 32) {
                const int r = i / DP, e = i % DP;
                const int row = row0 + 8 * n + r;
                if (row < P.rows && e < P.c.head_dim) {
                    const float *src = red + r * kRedRow + (e % (DP / 8)) / 2 * 16 + e / (DP / 8) * 2 + (e & 1);
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < WARPS; ++w) sum += src[w * 8 * kRedRow];
                    P.part_o[(slot * (NT * 8) + 8 * n + r) * P.c.head_dim + e] = sum;
                }
            }
            if (n + 1 < NT) __syncthreads();
        }
        for (int r = tid; r < NT * 8; r += WARPS * 32) {
            if (row0 + r >= P.rows) continue;
            float mx = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sh.m[w][r]);
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                if (sh.m[w][r] != -INFINITY) l += sh.l[w][r] * ex2(sh.m[w][r] - mx);
            // a token that is not there answers zero
            if (sh.word[(row0 + r) / P.group_heads] == 0) mx = -INFINITY, l = 0.f;
            float2 *ml = reinterpret_cast<float2 *>(P.part_ml) + slot * (NT * 8) + r;
            *ml = make_float2(mx, l);
        }
        __syncthreads();  // the next part overwrites queries, words and partial results
        at += gb - ga;
    }
}

// ---------------------------------------------------------------------------
// The parts of each row joined, rotated back, divided and rounded.  One CTA of
// four warps per row: the warps share the parts, warp 0 adds up and finishes.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 4;

template <int OT>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttnParams P, int tile_rows, int least) {
    __shared__ float so[kJoinWarps][256];
    __shared__ float sl[kJoinWarps];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x % P.rows;  // grid.x: rows of (sequence, head) pairs
    const int64_t bh = blockIdx.x / P.rows;
    const int b = (int)(bh / P.c.kv_heads), head = (int)(bh % P.c.kv_heads);
    const int tile = row / tile_rows, r = row % tile_rows;
    const int per_seq = P.c.kv_heads * P.row_tiles;
    const int64_t W = (int64_t)P.prefix[P.c.batch] * per_seq;
    const int ctas = cta_count(W, P.grid, least);
    const int hr = head * P.row_tiles + tile;
    const int groups = P.prefix[b + 1] - P.prefix[b];
    const int64_t first = (int64_t)P.prefix[b] * per_seq + (int64_t)hr * groups;
    // CTA of group x: the largest i with i W / ctas <= x
    const int64_t i0 = ((first + 1) * ctas - 1) / W, i1 = ((first + groups) * ctas - 1) / W;
    const int64_t unit = (int64_t)b * per_seq + hr;
    const float2 *ml = reinterpret_cast<const float2 *>(P.part_ml);

    float mx = -INFINITY;
    for (int64_t i = i0 + lane; i <= i1; i += 32) mx = fmaxf(mx, ml[(unit + i) * tile_rows + r].x);
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, k));
    const int D = P.c.head_dim;
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    float l = 0.f;
    for (int64_t i = i0 + warp; i <= i1; i += kJoinWarps) {
        const int64_t s = (unit + i) * tile_rows + r;
        const float2 p = ml[s];
        if (p.x == -INFINITY) continue;
        const float f = ex2(p.x - mx);
        l += f * p.y;
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
            const int e = sb * 128 + 4 * lane;
            if (e < D) {
                const float4 o = *reinterpret_cast<const float4 *>(P.part_o + s * D + e);
                acc[sb][0] += f * o.x;
                acc[sb][1] += f * o.y;
                acc[sb][2] += f * o.z;
                acc[sb][3] += f * o.w;
            }
        }
    }
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
        *reinterpret_cast<float4 *>(&so[warp][sb * 128 + 4 * lane]) =
            make_float4(acc[sb][0], acc[sb][1], acc[sb][2], acc[sb][3]);
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += sl[w];
    const float inv = l > 0.f ? 0.03125f / l : 0.f;
    const int t = row / P.group_heads, h = head * P.group_heads + row % P.group_heads;
    char *out = P.out + (b * P.o_batch + t * P.o_token + h * P.o_head) * ElemSize<OT>::value;
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
        const int e = sb * 128 + 4 * lane;
        if (sb * 128 >= D) break;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) v[i] += so[w][e + i];
            v[i] *= inv;
        }
        fwht32_warp(v, lane & 7);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = flip(v[i], sign_mask(e + i));
        if (e < D) store4<OT>(out + (int64_t)e * ElemSize<OT>::value, v);
    }
}

// Rows of a tile: 8, or 16 where a (sequence, head) has more than 8 rows and
// the accumulators of 16 fit the registers (head dimension up to 128).
struct AttnPlan {
    int dp, nt, warps, rows, row_tiles;
    int64_t units;
};

AttnPlan plan_attention(int64_t batch, int tree, int heads, int kv_heads, int head_dim) {
    AttnPlan p;
    p.dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
    p.rows = tree * (heads / kv_heads);
    p.nt = p.rows > 8 && p.dp <= 128 ? 2 : 1;
    p.warps = p.nt == 2 || p.dp == 256 ? 8 : 16;
    p.row_tiles = (p.rows + 8 * p.nt - 1) / (8 * p.nt);
    p.units = batch * kv_heads * p.row_tiles;
    return p;
}

template <int DP, int NT, int WARPS>
cudaError_t launch_attend(const AttnParams &P, cudaStream_t stream) {
    constexpr int bytes = attn_smem<DP, NT, WARPS>();
    static_assert(bytes <= kSmemLimit, "shared memory per CTA");
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<DP, NT, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bytes);
    if (e != cudaSuccess) return e;
    attend_kernel<DP, NT, WARPS><<<P.grid, WARPS * 32, bytes, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

size_t attention_workspace_bytes(int64_t batch, int tree, int heads, int kv_heads, int head_dim, int sm_count) {
    const AttnPlan p = plan_attention(batch, tree, heads, kv_heads, head_dim);
    const size_t slots = (size_t)(p.units + sm_count);
    return 256 + round_up((size_t)(batch + 1) * 4, 256) + round_up(slots * 8 * p.nt * 8, 256) +
           slots * 8 * p.nt * head_dim * 4;
}

cudaError_t launch_attention(const AttentionJob &j, int sm_count, cudaStream_t stream) {
    const AttnPlan plan = plan_attention(j.c.batch, j.tree, j.heads, j.c.kv_heads, j.c.head_dim);
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
    P.scale_log2 = j.scale * 1.44269504088896340736f;
    P.grid = sm_count;
    const size_t slots = (size_t)(plan.units + sm_count);
    char *ws = j.workspace + 256;
    P.prefix = reinterpret_cast<int *>(ws);
    ws += round_up((size_t)(j.c.batch + 1) * 4, 256);
    P.part_ml = reinterpret_cast<float *>(ws);
    ws += round_up(slots * 8 * plan.nt * 8, 256);
    P.part_o = reinterpret_cast<float *>(ws);

    cudaError_t e;
    if (plan.dp == 64) e = plan.nt == 1 ? launch_attend<64, 1, 16>(P, stream) : launch_attend<64, 2, 8>(P, stream);
    else if (plan.dp == 128) e = plan.nt == 1 ? launch_attend<128, 1, 16>(P, stream) : launch_attend<128, 2, 8>(P, stream);
    else e = launch_attend<256, 1, 8>(P, stream);
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)j.c.batch * j.c.kv_heads * plan.rows));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const int tile_rows = 8 * plan.nt, least = plan.warps;
    if (j.odtype == kF32) return cudaLaunchKernelEx(&cfg, join_kernel<kF32>, P, tile_rows, least);
    if (j.odtype == kBF16) return cudaLaunchKernelEx(&cfg, join_kernel<kBF16>, P, tile_rows, least);
    return cudaLaunchKernelEx(&cfg, join_kernel<kF16>, P, tile_rows, least);
}

}  // namespace tq
