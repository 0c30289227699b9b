// Elements of the 8-bit cache (e4m3: four significant bits down to 2^-6, a spacing
// of 2^-9 below, the largest 448, no infinities) and their scales.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace ple {
namespace {

// The least scale that the library writes: 2^kLeastExponent.
constexpr int kLeastExponent = -100;

// Two elements, the lower byte first, as halves; every element is a half exactly.
__device__ __forceinline__ uint32_t halves_of(uint16_t two) {
    uint32_t v;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"(two));
    return v;
}

// Four elements of a word as two pairs of halves.
__device__ __forceinline__ void halves_of(uint32_t four, uint32_t& low, uint32_t& high) {
    low = halves_of((uint16_t)four);
    high = halves_of((uint16_t)(four >> 16));
}

// Two values as elements, rounded to nearest, ties to even; past 448 they stay
// 448, and NaN is NaN.
__device__ __forceinline__ uint32_t elements_of(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

// Four elements under another scale.
__device__ __forceinline__ uint32_t scaled_elements(uint32_t w, float f) {
    uint32_t low, high;
    halves_of(w, low, high);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&low));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&high));
    return elements_of(a.x * f, a.y * f) | elements_of(b.x * f, b.y * f) << 16;
}

// Which of a word's four elements are NaN: their top bits.
__device__ __forceinline__ uint32_t nan_flags(uint32_t w) {
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// A scale (bfloat16) as a float.
__device__ __forceinline__ float scale_value(unsigned short bits) {
    return __uint_as_float((uint32_t)bits << 16);
}

// The exponent of the least power of two, at least 2^kLeastExponent, that takes a
// finite amount up to 448 of it: 448 is 1.75 * 2^8.
__device__ __forceinline__ int exponent_for(float most) {
    const uint32_t b = __float_as_uint(most);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, kLeastExponent);
}

}  // namespace
}  // namespace ple
