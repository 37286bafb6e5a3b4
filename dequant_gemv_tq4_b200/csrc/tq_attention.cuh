// tq_attention.cuh -- what the attention kernels share: the call's description,
// the split of the work, the ancestors of drafted tokens, the joining launch.
#pragma once

#include <math.h>

#include <type_traits>

#include "tq_cache.cuh"
#include "tq_internal.h"

namespace tq {

constexpr float kWeightExp = 7.0f;  // softmax weights are held times 2^7
constexpr float kLazy = 8.0f;       // log2 by which a maximum may grow before it is followed
constexpr float kNoMax = -1e30f;    // maximum of a row without a token so far (its sum is 0)

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
    float q_factor;    // scale log2(e) / 32: what a rotated query is multiplied with
    // the split and its results (workspace)
    int group;       // tokens of a group: what ranges are counted in
    int workers;     // ranges at most
    int least;       // groups of a range at least
    int extra;       // groups that beginning a unit counts for: its first `extra` hold no tokens
    int parts;       // partial results that a worker leaves of a unit
    int tile_rows;   // rows of a partial result
    unsigned *header;  // status word
    unsigned *status;  // [workers] each CTA's, of which the joining launch makes the header's; null: none reports
    long long timeout_cycles;  // of a wait in the tcgen05 kernel
    int inject_skip;           // test hook: the first tile's first keys are never handed over
    int inject_tmem;           // test hook: the last CTA takes its tensor memory for incomplete
    int *span;       // [units][2] first and last worker that leaves a part of the unit
    float *part_ml;  // [slots][tile_rows][2]: reference (log2), sum
    float *part_o;   // [slots][tile_rows][head_dim]
};

// Tokens that sequence b attends over, drafted ones included, within its table.
__device__ __forceinline__ int seq_tokens(const AttnParams &P, int len) {
    const int64_t cap = (int64_t)P.c.pages_per_seq << P.c.page_shift;
    const int64_t n = (int64_t)max(len, 0) + P.tree;
    return (int)(n < cap ? n : cap);
}

// The split of W groups: of n workers (warps or CTAs), worker i takes
// [i W / n, (i + 1) W / n), P.least groups or more.
__device__ __forceinline__ int worker_count(const AttnParams &P, int64_t W) {
    const int64_t n = (W + P.least - 1) / P.least;
    return (int)(n < P.workers ? n : P.workers);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The scale of a query row.  A row is multiplied with q_factor and a power of
// two that brings its largest element to [2^14, 2^15), whatever its size and the
// softmax's scale are: a rotated element is a mean of 32 and no larger, so it
// stays finite in fp16, and small rows keep their bits.  Scores s are then in
// units of a power of two, and under the running maximum m
//   weight = 2^(s unit + off),  off = fl(7 - m unit)
// is one fused operation at any size of the scores: m unit is exact, and where 7
// falls between the numbers that fp32 has there, it becomes one of 0 .. 8.  (With
// a factor that is no power of two the rounding of m times it alone would be many
// powers of two from 2^28 on.)  `off` stands for the maximum: sums and parts are
// referred to 2^-off, exactly.  `most`: the row's largest |element|; scores stay
// finite up to |q scale| = 2^40 and |q| = 2^122 (sums of 32), and a row beyond
// that, or with an infinity or a NaN, is all NaN, and so are its scores, sum and
// output.
struct RowScale {
    float factor;  // of the rotated query
    float unit;    // of the scores, in log2
    __device__ __forceinline__ RowScale(float q_factor, float most) {
        const float m = most * fabsf(q_factor) * 32.0f;
        const int e = min(max(14 + 127 - (int)(__float_as_uint(m) >> 23), -27), 90);
        const bool fits = m < 0x1p42f && most < 0x1p122f;
        factor = fits ? q_factor * __int_as_float((127 + e) << 23) : __int_as_float(0x7FFFFFFF);
        unit = __int_as_float((127 - e) << 23);
    }
};

// (finite for a row without a token so far, too: kNoMax times a unit of 2^27)
__device__ __forceinline__ float weight_offset(float m, float unit) { return fmaf(-m, unit, kWeightExp); }

// Whether a maximum mx is so far above the one that off stands for that it has
// to be followed: where its own weight would be above 2^15.
__device__ __forceinline__ bool outgrown(float mx, float unit, float off) {
    return fmaf(mx, unit, off) > kWeightExp + kLazy;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Which drafted tokens each drafted token sees, held by a warp: lane l has the
// words of tokens l and l + 32.  A word is the token itself and its ancestors,
// or 0 for a token that is not there (a parent that is neither -1 nor an
// earlier token, its own or an ancestor's).  Six rounds of pointer doubling.
struct TreeParents {
    int at[2];  // of tokens `lane` and `lane` + 32
    __device__ __forceinline__ TreeParents(const AttnParams &P, int b, int lane) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = lane + 32 * k;
            at[k] = P.parents && i < P.tree ? P.parents[b * P.parents_ld + i] : i - 1;
        }
    }
};

struct TreeWords {
    uint64_t w[2];
    __device__ __forceinline__ TreeWords(const AttnParams &P, const TreeParents &tree, int lane) {
        int ptr[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = lane + 32 * k;
            w[k] = i < P.tree ? (2ull << i) - 1 : 0;  // a chain
            ptr[k] = -1;
            if (P.parents && i < P.tree) {
                const int par = tree.at[k];
                ptr[k] = par < -1 || par >= i ? -2 : par;
                w[k] = 1ull << i;
            }
        }
        if (!P.parents || P.tree == 1) {
            if (ptr[0] == -2) w[0] = 0;
            return;
        }
        for (int hop = 1; hop < P.tree; hop <<= 1) {
            uint64_t nw[2];
            int np[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int from = ptr[k] & 31;
                const uint64_t a0 = __shfl_sync(kFull, w[0], from), a1 = __shfl_sync(kFull, w[1], from);
                const int p0 = __shfl_sync(kFull, ptr[0], from), p1 = __shfl_sync(kFull, ptr[1], from);
                nw[k] = w[k];
                np[k] = ptr[k];
                if (ptr[k] >= 0) {
                    nw[k] |= ptr[k] >= 32 ? a1 : a0;
                    np[k] = ptr[k] >= 32 ? p1 : p0;
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                w[k] = nw[k];
                ptr[k] = np[k];
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (ptr[k] == -2) w[k] = 0;
    }
    // word of token t (any per lane)
    __device__ __forceinline__ uint64_t of(int t) const {
        const uint64_t a0 = __shfl_sync(kFull, w[0], t & 31), a1 = __shfl_sync(kFull, w[1], t & 31);
        return t >= 32 ? a1 : a0;
    }
    // bit t: token t is there
    __device__ __forceinline__ uint64_t present() const {
        return (uint64_t)__ballot_sync(kFull, w[0] != 0) | ((uint64_t)__ballot_sync(kFull, w[1] != 0) << 32);
    }
};

// Exclusive prefix of the sequences' groups into `prefix`, by the whole CTA.
__device__ __forceinline__ void scan_sequences(const AttnParams &P, int *prefix, int *scan, int tid, int threads) {
    const int per = (P.c.batch + threads - 1) / threads;
    int sum = 0;
    for (int i = tid * per; i < min(P.c.batch, (tid + 1) * per); ++i)
        sum += (seq_tokens(P, P.lens[i]) + P.group - 1) / P.group + P.extra;
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
        at += (seq_tokens(P, P.lens[i]) + P.group - 1) / P.group + P.extra;
    }
    if (tid == threads - 1) prefix[P.c.batch] = base + inc;
    __syncthreads();
}

// The launch that joins the parts of every row, rotates back, divides and
// rounds; a programmatic dependent of the attention launch before it.
cudaError_t launch_join(const AttnParams &P, int odtype, cudaStream_t stream);

// The tcgen05 kernel (tq_tcattention.cu): tiles of 128 or 256 rows.
bool tc_attention_fits(int head_dim);
cudaError_t launch_tc_attention(const AttnParams &P, cudaStream_t stream);
int tc_attention_tile_rows(int rows);

}  // namespace tq
