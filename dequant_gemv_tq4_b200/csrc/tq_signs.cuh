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

}  // namespace tq
