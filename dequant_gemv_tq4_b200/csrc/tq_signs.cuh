// tq_signs.cuh -- the sign pattern of a head's columns as a constant table, for
// the key/value cache and the attention over it (heads of up to 256 elements).
#pragma once

#include <stdint.h>

namespace tq {

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

}  // namespace tq
