// Rows in 8 bits: the scale of a row and the codes of its elements, as the
// state cache and the norm form them.
#pragma once

#include "ssd_common.hpp"

namespace ssd {

// x / s to the nearest integer, ties to even, decided on the true quotient:
// the product with the rounded reciprocal is within one of it, and the
// remainder x - c s is exact in fp32 (a multiple of half a unit of s's last
// place, below s in size).
__device__ __forceinline__ int nearest_code(float x, float s, float inv) {
    float c = rintf(x * inv);
    const float r = 2.f * __builtin_fmaf(-c, s, x);
    const float a = fabsf(r);
    const bool odd = ((int)c & 1) != 0;
    if (a > s || (a == s && odd)) c += r > 0.f ? 1.f : -1.f;
    return (int)c;
}

// top / 127, correctly rounded: by Markstein's theorem one step from a product
// with the rounded reciprocal gives it, away from the subnormal range.
__device__ __forceinline__ float code_scale(float top) {
    constexpr float inv = 1.f / 127.f;
    if (top < 0x1p-100f) return top / 127.f;
    const float q = top * inv;
    return __builtin_fmaf(__builtin_fmaf(-127.f, q, top), inv, q);
}

// Biased exponent of the scale of an e4m3 row whose largest magnitude has
// these bits: top = m 2^e, and 448 = 1.75 2^8 holds m <= 1.75 with 2^(e-8).
__device__ __forceinline__ int e4m3_scale_exponent(uint32_t top) {
    const int k = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return k < 1 ? 1 : k;
}

}  // namespace ssd
