// kda_cache.cuh -- the paged 8-bit cache: its layout and its numbers.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "kda_common.cuh"

namespace kda {

// A page holds `page` tokens (a power of two) of every head:
//   codes  [n_pages][H][page][d] e4m3        scale [n_pages][H] fp32
// value = code * scale; a scale is a power of two, so that a value is scaled
// and moved from one scale to another without rounding (but for codes that go
// below e4m3's normal range).
constexpr float kE4m3Max = 448.0f;
constexpr int kScaleMinExp = -100;   // the scale of a page that holds only zeros

// The least power of two, from 2^kScaleMinExp up, that brings a finite
// amax >= 0 to 448 = 1.75 * 2^8 or less.  Exponent arithmetic on the bits:
// amax = m 2^x with 1 <= m < 2 needs x - 8, or x - 7 where m > 1.75.
__device__ __forceinline__ float page_scale(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < kScaleMinExp ? kScaleMinExp : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
// A page's scale as read back, if it is positive and in the range that page_scale gives;
// else 0 (a page that was never written), whose codes then count for nothing.
__device__ __forceinline__ float valid_scale(float s) {
    return s >= 7.888609052210118e-31f && s <= 1.329227995784916e36f ? s : 0.0f;   // 2^-100, 2^120
}
// The least power of two that is no less.
__device__ __forceinline__ float pow2_ceil(float s) {
    return __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0xff800000u);
}
// 1 / s of a power of two in [2^-126, 2^126].
__device__ __forceinline__ float pow2_inverse(float s) {
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// |x| where x is finite, 0 otherwise: infinities and NaN set no scale.
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.4028234663852886e38f ? a : 0.0f;
}

// Four values to four codes: nearest, ties to even; what is above 448 (an
// infinity) becomes 448, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
// Two codes (the low 16 bits) to two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(two));
    return h;
}
__device__ __forceinline__ void from_e4m3x4(uint32_t four, float* f) {
    const uint32_t lo = e4m3x2_to_half2(four & 0xffffu), hi = e4m3x2_to_half2(four >> 16);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

}  // namespace kda
