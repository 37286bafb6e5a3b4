// tq_cache.cuh -- what the key/value cache's kernels and the attention over it
// share: the sign pattern of a head's columns, and a 32-element block in one
// lane's registers, with the arithmetic of the weight codec (tq_codec.cu),
// operation for operation.
#pragma once

#include "tq_device.cuh"

namespace tq {

// a / b of non-negative numbers, in 32 bits where both fit
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The codec's signs of the head's columns, a bit per column (1 = negative).
struct SignWords {
    uint32_t w[8];
};
constexpr SignWords sign_words() {
    SignWords s = {};
    for (uint32_t k = 0; k < 256; ++k) {
        uint32_t h = k * 0x9E3779B9u;
        h ^= h >> 16;
        h *= 0x85EBCA6Bu;
        h ^= h >> 13;
        s.w[k / 32] |= (h >> 31) << (k % 32);
    }
    return s;
}
static __constant__ SignWords c_sign_words = sign_words();

// The same for pairs of 16-bit values: word b has the signs of block b's even
// columns in its low half and of the odd ones in its high half, so that one
// shift brings column pair i to bits 15 and 31.
constexpr SignWords sign_pairs() {
    const SignWords s = sign_words();
    SignWords p = {};
    for (int b = 0; b < 8; ++b)
        for (int i = 0; i < 16; ++i)
            p.w[b] |= ((s.w[b] >> (2 * i)) & 1u) << i | ((s.w[b] >> (2 * i + 1)) & 1u) << (16 + i);
    return p;
}
static __constant__ SignWords c_sign_pairs = sign_pairs();

// Code of one rotated value y against the ascending thresholds t of its half,
// added into `word` at nibble position `sh`: bit 3 = [y < 0], bits 0..2 =
// #{j : |y| > t_j} by a three-compare binary search.  Each bit is a
// conditional add consumed right after its compare, so the compiler can
// predicate the adds instead of materialising (or spilling) the predicates.
__device__ __forceinline__ uint32_t add_code(uint32_t word, float y, const float (&t)[7], int sh) {
    const float a = fabsf(y);
    const bool b2 = a > t[3];
    const bool b1 = a > (b2 ? t[5] : t[1]);
    const bool b0 = a > (b1 ? (b2 ? t[6] : t[2]) : (b2 ? t[4] : t[0]));
    if (b2) word += 4u << sh;
    if (b1) word += 2u << sh;
    if (b0) word += 1u << sh;
    if (y < 0.0f) word += 8u << sh;
    return word;
}

// Packed fp32 pairs (sm_100 add/sub.rn.f32x2): each half is one IEEE fp32
// operation rounded to nearest even, exactly the scalar __fadd_rn/__fsub_rn.
// Their operands here are loads or scalar products, never a packed product
// (a packed multiply feeding a packed add may be contracted into an FMA).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The 32-point transform in the codec's stage order h = 1, 2, 4, 8, 16.
// Element t and element t + 16 share one packed register: stages h < 16 pair
// register t with register t + h (both halves at once), stage 16 combines
// the two halves of each register in scalar.  Every element sees the same
// operations on the same operands as the sequential definition.
__device__ __forceinline__ void fwht32_regs(float (&v)[32]) {
    uint64_t P[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) P[t] = pack2(v[t], v[t + 16]);
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if ((i & h) == 0) {
                const uint64_t a = P[i], b = P[i + h];
                P[i] = add2(a, b);
                P[i + h] = sub2(a, b);
            }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
        float lo, hi;
        unpack2(P[t], lo, hi);
        v[t] = __fadd_rn(lo, hi);
        v[t + 16] = __fsub_rn(lo, hi);
    }
}

}  // namespace tq
