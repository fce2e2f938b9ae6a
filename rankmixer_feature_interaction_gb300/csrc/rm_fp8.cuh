// Device helpers of the 8-bit operators: the block exponent, codes and their
// values (the format of include/rankmixer.h, "8-bit operands and checkpoints").
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rm_common.cuh"
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

// Largest of three (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Gelu(u) = u Phi(u) for the epilogues that hold a row in registers, written as
// relu(u) - |u| Q(|u|) with the upper tail Q = 1 - Phi.  Q is positive and its
// logarithm nearly a parabola, so one exponential of a polynomial gives it,
// Q(x) = 2^P(x): P of degree 7 fitted to log2 Q over [0, 12.9] (where Q is the
// smallest normal float) by a linear program, for the smallest largest error in Q,
// 2.4e-7, under the condition that Q is within 1.5% of itself everywhere: a block
// of 8-bit outputs is scaled by its own largest value, so where all of its u are far
// below zero the tail's relative error is what is kept (half a step is 6%).
// P falls for all x (its leading coefficient is negative) and the exponential
// flushes below 2^-126, so Gelu goes to zero without a bound on x.  In float32 the
// result is within 3.5e-7 |u|.  Ten instructions, every constant an immediate of
// its own (the rational form needs a reciprocal and an exponential; the packed
// two-value form needs constants in register pairs, for which 64 held values leave
// no room).
__device__ __forceinline__ float fp8_gelu(float u) {
    const float x = fabsf(u);
    float p = fmaf(x, -9.30538079e-07f, 4.20015094e-05f);
    p = fmaf(x, p, -7.80347327e-04f);
    p = fmaf(x, p, 8.01421981e-03f);
    p = fmaf(x, p, -5.32146059e-02f);
    p = fmaf(x, p, -4.58957642e-01f);
    p = fmaf(x, p, -1.15113652f);
    p = fmaf(x, p, -9.99999404e-01f);
    return fmaf(-x, ex2_approx(p), fmaxf(u, 0.f));
}

// Gelu'(u) = Phi(u) + u phi(u), by Abramowitz & Stegun 7.1.26 (|error of erf| <=
// 1.5e-7) as in rm_common.cuh, with phi(u) = exp(-u^2 / 2) / sqrt(2 pi).
__device__ __forceinline__ float fp8_gelu_grad(float u) {
    const float t = rcp_approx(fmaf(fabsf(u), 0.23164189f, 1.0f));   // p / sqrt 2
    float q = fmaf(t, 0.5307027145f, -0.7265760135f);                // a_i / 2
    q = fmaf(t, q, 0.7107068705f);
    q = fmaf(t, q, -0.142248368f);
    q = fmaf(t, q, 0.127414796f);
    const float e = ex2_approx(u * u * -0.72134752f);                // log2(e) / 2
    return fmaf(u * 0.39894228f, e, 0.5f + copysignf(0.5f - q * t * e, u));
}

}  // namespace rm
