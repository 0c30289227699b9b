// Elements of the 8-bit cache (e4m3: four significant bits down to 2^-6, a spacing
// of 2^-9 below, the largest 448, no infinities) and their scales.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ple.h"

namespace ple {
namespace {

// The least scale that the library writes: 2^kLeastExponent.
constexpr int kLeastExponent = -100;
constexpr int kMostBlock = 128;    // slots under one scale

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

// Four elements kept under a scale that is `f + rest` of the new one, f of 20 significant bits
// and rest >= 0 (a zero keeps its sign): e * f is exact, so that a quotient on the border of two
// elements, which one factor of 24 bits may miss, is met there.  Any other is 2^-13 of itself
// away from it.
__device__ __forceinline__ uint32_t scaled_elements(uint32_t w, float f, float rest) {
    uint32_t low, high;
    halves_of(w, low, high);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&low));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&high));
    return elements_of(fmaf(a.x, rest, a.x * f), fmaf(a.y, rest, a.y * f)) |
           elements_of(fmaf(b.x, rest, b.x * f), fmaf(b.y, rest, b.y * f)) << 16;
}

// What takes a scale to [1, 2), the least ones, which are no normal numbers, to below that: so
// quotients of scales, and what is left of them, stay inside 32 bits.
__device__ __forceinline__ float scale_to_one(float scale) {
    const uint32_t e = __float_as_uint(scale) >> 23;
    return e < 254 ? __uint_as_float((254 - e) << 23) : 0x1p-127f;
}

// The same where infinities are NaN too.
__device__ __forceinline__ uint32_t nearest_elements(float lo, float hi) {
    lo = fabsf(lo) < INFINITY ? lo : __int_as_float(0x7FC00000);
    hi = fabsf(hi) < INFINITY ? hi : __int_as_float(0x7FC00000);
    return elements_of(lo, hi);
}

// Which of a word's four elements are NaN: their top bits.
__device__ __forceinline__ uint32_t nan_flags(uint32_t w) {
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// A scale (bfloat16) as a float.
__device__ __forceinline__ float scale_value(uint32_t bits) {
    return __uint_as_float(bits << 16);
}

// log2 of a scale (the bits of a bfloat16), exact for a power of two, and finite whatever
// it is.
__device__ __forceinline__ float scale_log(uint32_t bits) {
    const float scale = scale_value(bits);
    if ((bits & 0x7F) == 0 && bits - 0x80 < 0x7F00) return (float)((int)(bits >> 7) - 127);
    float l;
    asm("lg2.approx.f32 %0, %1;" : "=f"(l) : "f"(scale));
    return fminf(fmaxf(l, -1000.f), 1000.f);
}

// Loads that are issued where they stand: what asks ahead is not moved to where its
// answer is used.
// (Into a whole register: two of 16 bits would be put into one, behind the loads.)
__device__ __forceinline__ uint32_t load_now(const unsigned short* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int load_now(const int* p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// Where the attention kernels find scales.
struct Scales {
    const unsigned short *k, *v;
    int64_t page, head;       // strides
    int32_t shift;            // log2 of a block's tokens
    // x / page_size below 2^31 as (x + high word of x * page_magic) >> page_shift: division
    // by a constant (Granlund and Montgomery 1994)
    uint32_t page_magic;
    int32_t page_shift;

    __device__ __forceinline__ uint32_t page_of(uint32_t slot) const {
        return (__umulhi(slot, page_magic) + slot) >> page_shift;
    }
    __device__ __forceinline__ int in_page(uint32_t slot, int page_size) const {
        return (int)(slot - page_of(slot) * page_size);
    }

    // Asks for the scales of a slot's keys and values, its page being `number` of `pages` (of
    // any other: 1).  Nothing here waits for them.
    __device__ __forceinline__ void ask(int number, int64_t pages, int of_head, uint32_t slot,
                                        int page_size, uint32_t& of_keys,
                                        uint32_t& of_values) const {
        of_keys = of_values = 0x3F80;
        if (number < 0 || number >= pages) return;
        const int64_t at = number * page + of_head * head +
                           ((slot - page_of(slot) * page_size) >> shift);
        of_keys = load_now(k + at);
        of_values = load_now(v + at);
    }
};

inline int block_shift(int block) {
    return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
}

inline Scales scales_of(const ple_tree_attention_fp8_args& f) {
    Scales s;
    s.k = static_cast<const unsigned short*>(f.scales.k);
    s.v = static_cast<const unsigned short*>(f.scales.v);
    s.page = f.scales.page_stride;
    s.head = f.scales.head_stride;
    s.shift = block_shift(f.scales.block);
    // with l bits of the divisor d: floor(2^32 (2^l - d) / d) + 1
    const uint64_t d = f.base.page_size;
    int l = 0;
    while ((uint64_t)1 << l < d) ++l;
    s.page_shift = l;
    s.page_magic = (uint32_t)(((uint64_t)1 << 32) * (((uint64_t)1 << l) - d) / d + 1);
    return s;
}

// The exponent of the least power of two, at least 2^kLeastExponent, that takes a
// finite amount up to 448 of it: 448 is 1.75 * 2^8.
__device__ __forceinline__ int exponent_for(float most) {
    const uint32_t b = __float_as_uint(most);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(e, kLeastExponent);
}

// A row's queries as sums of elements: times 2^-shift, so that the largest is in
// [128, 256).
__device__ __forceinline__ int term_shift(float most) {
    const int e = (int)(__float_as_uint(most) >> 23) - 127;
    return e > 127 ? 0 : max(e - 7, -100);
}

// Two 16-bit values of a word.
template <bool kBf16>
__device__ __forceinline__ void widen_pair(uint32_t v, float& lo, float& hi) {
    if constexpr (kBf16) {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xFFFF0000u);
    } else {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v));
        lo = x.x;
        hi = x.y;
    }
}

// A row's queries as halves: those of float16 as they are, those of bfloat16 times
// 2^-shift so that the largest is near 2^15: the rest lose what lies below 2^-40 of it.
__device__ __forceinline__ int query_shift(uint32_t most) {
    const int e = (int)(most >> 23) - 127;
    return e > 127 ? 0 : max(e - 14, -100);
}

}  // namespace
}  // namespace ple
