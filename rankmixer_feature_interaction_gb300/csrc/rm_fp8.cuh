// Device helpers of the 8-bit operators: the block exponent, codes and their
// values (the format of include/rankmixer.h, "8-bit operands and checkpoints").
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rm_fp8.h"

namespace rm {

// Exponent byte of a block whose largest finite magnitude has the float bits
// amax: the smallest E with amax <= 0.875 2^top 2^(E - 127) (0.875 2^top is the
// format's largest value: 448 = 0.875 2^9, 57344 = 0.875 2^16).  With amax =
// 1.m 2^(x - 127) that is E = x + 1 - top, one more when 1.m > 1.75.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_exponent(uint32_t amax) {
    constexpr int top = E5M2 ? 16 : 9;
    if (amax == 0u) return 127u;
    const int e = (int)(amax >> 23) + 1 - top + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 1 ? 1 : e);
}

// 2^(127 - E) for E in [1, 253]: what values are multiplied by before rounding.
__device__ __forceinline__ float fp8_inv_scale(uint32_t E) { return __uint_as_float((254u - E) << 23); }

// 2^(E - 127) for any byte (255: NaN; 0: 2^-127, a subnormal float).
__device__ __forceinline__ float fp8_scale(uint32_t E) {
    return E == 0u ? __uint_as_float(0x00400000u) : E == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(E << 23);
}

// Two floats (already scaled) to two codes, lo in the low byte; NaN to a NaN code.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_pack2(float lo, float hi) {
    uint16_t r;
    if (E5M2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    return fp8_pack2<E5M2>(a, b) | (fp8_pack2<E5M2>(c, d) << 16);
}

// Two codes to the two numbers they stand for (exact).
template <bool E5M2>
__device__ __forceinline__ float2 fp8_unpack2(uint32_t codes) {
    uint32_t h;
    const uint16_t c = (uint16_t)codes;
    if (E5M2)
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
    else
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ uint32_t fp8_finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// Infinities become NaN (the code for both).
__device__ __forceinline__ float fp8_poison(float x) {
    return (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u ? x : __uint_as_float(0x7fc00000u);
}

}  // namespace rm
