// Device helpers of the 4-bit operators: the block exponent, codes and their
// values (the format of include/rankmixer.h, "4-bit operands").
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rm_common.cuh"
#include "rm_fp4.h"

namespace rm {

// Exponent byte of a block whose largest magnitude has the float bits amax: the
// smallest E with amax <= 6 2^(E - 127), at least 1; 127 for zeros; 255 (the block
// is NaN) where a value is not finite.  6 = 1.5 2^2, so with amax = 1.m 2^(x - 127)
// that is E = x - 2, one more when 1.m > 1.5.
__device__ __forceinline__ uint32_t fp4_exponent(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255u;
    const int e = (int)(amax >> 23) - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0);
    return amax == 0u ? 127u : (uint32_t)(e < 1 ? 1 : e);
}
// 2^(127 - E) for E in [1, 253]; 0 for 255.
__device__ __forceinline__ float fp4_inv_scale(uint32_t E) { return E == 255u ? 0.f : __uint_as_float((254u - E) << 23); }

// Eight floats (already scaled) to eight codes, the first in the lowest bits: to the
// nearest, ties to the even code.
__device__ __forceinline__ uint32_t fp4_pack8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// The eight numbers that eight codes stand for (exact).
__device__ __forceinline__ void fp4_unpack8(uint32_t codes, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t fp4_abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Largest of three; NaN where one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Sixteen values of a row as they lie in memory, zeros past its end.
template <typename IN>
struct Fp4Raw16 {
    static constexpr int WORDS = 4 * sizeof(IN);
    uint32_t w[WORDS];
    // VEC: p is 16-byte aligned where n is 16 or more
    template <bool VEC>
    __device__ __forceinline__ void load(const IN* __restrict__ p, int n) {
        if (VEC && n >= 16) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                if constexpr (sizeof(IN) == 4) {
                    w[i] = i < n ? __float_as_uint(p[i]) : 0u;
                } else {
                    w[i] = 2 * i < n ? __bfloat16_as_ushort(p[2 * i]) : 0u;
                    if (2 * i + 1 < n) w[i] |= (uint32_t)__bfloat16_as_ushort(p[2 * i + 1]) << 16;
                }
            }
        }
    }
    // Any row, the values from X[at] on: the whole 16-byte pieces of memory around them,
    // shifted into place; one by one where those might leave X, which has `size` values.
    __device__ __forceinline__ void load_any(const IN* __restrict__ X, unsigned long long at, int n, unsigned long long size) {
        constexpr int AROUND = 16 / (int)sizeof(IN);
        const IN* p = X + at;
        constexpr int ESZ = sizeof(IN);
        if (n <= 0 || at < AROUND || at + 16 + AROUND > size) {
            load<false>(p, n);
            return;
        }
        const uint32_t o = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u, bytes = o + ESZ * min(n, 16);
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - o);
        uint32_t t[WORDS + 4];
#pragma unroll
        for (int i = 0; i <= WORDS / 4; ++i) {
            const uint4 x = 16u * i < bytes ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
            t[4 * i] = x.x, t[4 * i + 1] = x.y, t[4 * i + 2] = x.z, t[4 * i + 3] = x.w;
        }
        if (o & 8) {
#pragma unroll
            for (int i = 0; i + 2 < WORDS + 4; ++i) t[i] = t[i + 2];
        }
        if (o & 4) {
#pragma unroll
            for (int i = 0; i + 1 < WORDS + 4; ++i) t[i] = t[i + 1];
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = ESZ == 4 ? t[i] : __funnelshift_r(t[i], t[i + 1], 8 * (o & 2));
        if (n < 16) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                if (4 * i >= ESZ * n) w[i] = 0;
                if (4 * i + 2 >= ESZ * n) w[i] &= 0xffffu;
            }
        }
    }
    // float bits of the largest magnitude; infinities and NaN count as they are
    __device__ __forceinline__ uint32_t amax_bits() const {
        uint32_t m = 0;
        if constexpr (sizeof(IN) == 2) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            return max(m << 16, m & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        }
    }
    __device__ __forceinline__ uint32_t codes(int half, uint64_t scale) const {
        float q[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t pair;
            if constexpr (sizeof(IN) == 2) {
                const uint32_t x = w[4 * half + i];
                pair = f2_pack(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
            } else {
                pair = f2_pack(__uint_as_float(w[8 * half + 2 * i]), __uint_as_float(w[8 * half + 2 * i + 1]));
            }
            f2_unpack(f2_mul(pair, scale), q[2 * i], q[2 * i + 1]);
        }
        return fp4_pack8(q);
    }
    // Codes, by the scale of the block that this lane and its neighbour (lane ^ 1) hold.
    __device__ __forceinline__ uint2 round(uint32_t& E) const {
        uint32_t m = amax_bits();
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        E = fp4_exponent(m);
        const uint64_t s = f2_splat(fp4_inv_scale(E));
        return make_uint2(codes(0, s), codes(1, s));
    }
};

}  // namespace rm
