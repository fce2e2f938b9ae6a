// Elementwise kernels of the 8-bit operators: saving rows and weights in 8 bits,
// and restoring rows.
//
// Saving reads every value once and writes one byte for it; 8 lanes own one block
// of 128 values, two runs of 8 each (a load instruction's 8 lanes read 128 bytes
// in a row), agree on its largest magnitude with three shuffles and write twice 8
// bytes of codes.  64 bytes per thread are loaded before the first is used and stay
// as they came (bf16 pairs) until then: few registers, so many warps, are what
// hides the loads' latency, and few instructions per value what lets them.  Rows
// that are not 16-byte aligned are read an element at a time, neighbouring lanes
// neighbouring elements, and their codes pass through shared memory to the same
// 8-byte stores; restoring such rows mirrors that.
// Measured, 65,536 rows of 6144 in bf16 (805 MB; 406 MB in 8 bits): saving 185 us,
// restoring 185 us, 6.5 TB/s each: bound by memory.  6185 rows of 1003 in float32,
// which are not 16-byte aligned, to e5m2 and bf16: 8.0 and 9.3 us (25 and 19 MB; of 1008,
// aligned, 4.4 and 6.2).  302 M weights: from float32 208 us (7.2 TB/s), from bf16 286.
#include <type_traits>

#include "rm_common.cuh"
#include "rm_fp8.cuh"

namespace rm {
namespace {

constexpr int kThreads = 256;
// 16-byte pieces of codes in flight per thread when restoring: 805 MB in bf16 took
// 185 us with 2, 205 with 4, 253 with 8 (the pieces' stores queue behind each other).
constexpr int kUnroll = 2;

template <typename IN, bool VEC>
__device__ __forceinline__ void load8(const IN* __restrict__ p, int n, float (&v)[8]) {
    if (VEC && n >= 8) {
        if constexpr (sizeof(IN) == 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        } else {
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
    }
}

// Row and piece (of n per row) of a running number, and of the one `step` further
// (step = dq n + dr).
__device__ __forceinline__ void split_id(unsigned long long id, unsigned long long count, int n, unsigned long long& row,
                                         int& j) {
    if (count <= 0xffffffffull) {
        const uint32_t r = (uint32_t)id / (uint32_t)n;
        row = r;
        j = (int)((uint32_t)id - r * (uint32_t)n);
    } else {
        row = id / (unsigned)n;
        j = (int)(id - row * (unsigned)n);
    }
}
__device__ __forceinline__ void next_id(unsigned long long& row, int& j, int dq, int dr, int n) {
    row += dq;
    j += dr;
    if (j >= n) j -= n, ++row;
}

// Eight values of a row as they lie in memory, zeros past its end.
template <typename IN>
struct Raw8 {
    uint32_t w[sizeof(IN) * 2];
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(IN) == 2)
            return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        else
            return __uint_as_float(w[i]);
    }
    __device__ __forceinline__ void set(int i, IN x) {
        if constexpr (sizeof(IN) == 2)
            w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | ((uint32_t)__bfloat16_as_ushort(x) << 16)
                              : (w[i >> 1] & 0xffff0000u) | __bfloat16_as_ushort(x);
        else
            w[i] = __float_as_uint(x);
    }
    __device__ __forceinline__ void load(const IN* __restrict__ p, int n) {
        if (n >= 8) {
#pragma unroll
            for (int k = 0; k < (int)sizeof(IN) / 2; ++k) {
                const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + k);
                w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(IN) * 2; ++i) w[i] = 0;
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) set(i, p[i]);
        }
    }
    // every eighth value from p on, 8 of them
    __device__ __forceinline__ void gather(const IN* __restrict__ p, int n) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(IN) * 2; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (8 * i < n) set(i, p[8 * i]);
    }
    // float bits of the largest magnitude; infinities and NaN count as they are
    __device__ __forceinline__ uint32_t amax_bits() const {
        uint32_t m = 0;
        if constexpr (sizeof(IN) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            return max(m << 16, m & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        }
    }
};

// Blocks per 8 lanes: 64 bytes of values per thread.
template <typename IN>
constexpr int kBlocks = sizeof(IN) == 2 ? 2 : 1;

template <typename IN, bool E5M2, bool VEC, bool COPY>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const IN* __restrict__ X, unsigned long long blocks, int cols, int nb, int dq, int dr, long long ldx,
                Fp8View out, __nv_bfloat16* __restrict__ copy) {
    static_assert(VEC || !COPY, "the copy takes eight neighbouring values of a lane");
    constexpr int UNROLL = kBlocks<IN>, PER = kThreads / 8;
    __shared__ uint2 bytes[VEC ? 1 : 2 * kThreads];  // a block's 128 codes are contiguous
    pdl_wait();
    pdl_launch_next();
    const int l8 = threadIdx.x & 7;
    const unsigned long long base = (unsigned long long)blockIdx.x * (PER * UNROLL) + (threadIdx.x >> 3);
    Raw8<IN> v[UNROLL][2];
    unsigned long long row0 = 0;
    int j0 = 0;
    if (base < blocks) split_id(base, blocks, nb, row0, j0);
    {
        unsigned long long row = row0;
        int j = j0;
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int n = base + (unsigned long long)i * PER < blocks ? cols - j * kFp8Block : 0;
            const IN* p = X + row * (unsigned long long)ldx + j * kFp8Block;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (VEC)
                    v[i][h].load(p + 8 * l8 + 64 * h, n - 8 * l8 - 64 * h);
                else
                    v[i][h].gather(p + l8 + 64 * h, n - l8 - 64 * h);
            }
            next_id(row, j, dq, dr, nb);
        }
    }
    unsigned long long row = row0;
    int j = j0;
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
        uint32_t m = max(v[i][0].amax_bits(), v[i][1].amax_bits());
        const bool odd = m >= 0x7f800000u;           // infinities or NaN among them: neither counts
        if (odd) {
            m = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) m = max(m, fp8_finite_bits(v[i][h].get(k)));
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t E = fp8_exponent<E5M2>(m);
        const uint64_t s = f2_splat(fp8_inv_scale(E));
        uint2 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; k += 2)
                f2_unpack(f2_mul(f2_pack(v[i][h].get(k), v[i][h].get(k + 1)), s), f[k], f[k + 1]);
            if (odd) {                               // infinities become NaN
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = fp8_poison(v[i][h].get(k)) * fp8_inv_scale(E);
            }
            w[h] = make_uint2(fp8_pack4<E5M2>(f[0], f[1], f[2], f[3]), fp8_pack4<E5M2>(f[4], f[5], f[6], f[7]));
        }
        if (!VEC) {                                  // lane's codes are every eighth: to their places
            uint2* block = bytes + (threadIdx.x & ~7) * 2;
            uint8_t* mine = reinterpret_cast<uint8_t*>(block) + l8;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) mine[64 * h + 8 * k] = (uint8_t)((k < 4 ? w[h].x : w[h].y) >> (8 * (k & 3)));
            __syncwarp();
            w[0] = block[l8];
            w[1] = block[8 + l8];
            __syncwarp();
        }
        if (base + (unsigned long long)i * PER < blocks) {
            if (l8 == 0) out.scales[row * (unsigned long long)out.lds + j] = (uint8_t)E;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = j * kFp8Block + 8 * l8 + 64 * h;
                // code rows are padded to 16 bytes, so a lane's 8 fit when they begin before that
                if (col < (cols + 15) / 16 * 16) {
                    *reinterpret_cast<uint2*>(out.codes + row * (unsigned long long)out.ld + col) = w[h];
                    if (COPY)                        // cols is a multiple of 16
                        *reinterpret_cast<uint4*>(copy + row * (unsigned long long)cols + col) =
                            make_uint4(pack_bf16x2(v[i][h].get(0), v[i][h].get(1)), pack_bf16x2(v[i][h].get(2), v[i][h].get(3)),
                                       pack_bf16x2(v[i][h].get(4), v[i][h].get(5)), pack_bf16x2(v[i][h].get(6), v[i][h].get(7)));
                }
            }
        }
        next_id(row, j, dq, dr, nb);
    }
}

// One CTA per 128 x 128 block of a token's weight: 16 rows x 16 lanes of 8
// columns at a time, all 64 values of a thread kept for the second half.
template <typename IN, bool VEC>
__global__ void __launch_bounds__(kThreads)
quantize_weight_kernel(const IN* __restrict__ W, int K, int N, Fp8View out) {
    __shared__ uint32_t part[kThreads / 32];
    pdl_wait();
    pdl_launch_next();
    const int kb = blockIdx.y, t = blockIdx.z, c0 = blockIdx.x * kFp8Block + 8 * (threadIdx.x & 15);
    float v[8][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = kb * kFp8Block + 16 * i + (threadIdx.x >> 4);
        load8<IN, VEC>(W + ((size_t)t * K + (k < K ? k : 0)) * N + c0, k < K ? N - c0 : 0, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, fp8_finite_bits(v[i][j]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, part[w]);
    const uint32_t E = fp8_exponent<false>(m);
    const float s = fp8_inv_scale(E);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = kb * kFp8Block + 16 * i + (threadIdx.x >> 4);
        if (k < K && c0 < (N + 15) / 16 * 16) {
            float q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = fp8_poison(v[i][j]) * s;
            *reinterpret_cast<uint2*>(out.codes + ((size_t)t * K + k) * out.ld + c0) =
                make_uint2(fp8_pack4<false>(q[0], q[1], q[2], q[3]), fp8_pack4<false>(q[4], q[5], q[6], q[7]));
        }
    }
    if (threadIdx.x == 0) out.scales[((size_t)t * gridDim.y + kb) * out.lds + blockIdx.x] = (uint8_t)E;
}

template <typename OUT, bool E5M2, bool VEC>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(Fp8View in, unsigned long long chunks, int cols, int nch, int dq, int dr, OUT* __restrict__ Y,
                  long long ldy) {
    // one thread per 16 codes, kUnroll chunks in flight
    __shared__ OUT stage[VEC ? 1 : kThreads * 17];   // a thread's 16 values, one apart from the next thread's
    pdl_wait();
    pdl_launch_next();
    const unsigned long long base = (unsigned long long)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint4 w[kUnroll];
    float sc[kUnroll];
    unsigned long long row[kUnroll];
    int col[kUnroll];
    unsigned long long r = 0;
    int c = 0;
    if (base < chunks) split_id(base, chunks, nch, r, c);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        row[i] = r;
        col[i] = cols;
        w[i] = make_uint4(0, 0, 0, 0);
        sc[i] = 0.f;
        if (base + (unsigned long long)i * kThreads < chunks) {
            col[i] = 16 * c;
            w[i] = __ldcs(reinterpret_cast<const uint4*>(in.codes + r * (unsigned long long)in.ld + col[i]));
            sc[i] = fp8_scale(in.scales[r * (unsigned long long)in.lds + col[i] / kFp8Block]);
        }
        next_id(r, c, dq, dr, nch);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int n = cols - col[i];
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float v[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 f = fp8_unpack2<E5M2>(u[k >> 1] >> (16 * (k & 1)));
            v[2 * k] = f.x * sc[i];
            v[2 * k + 1] = f.y * sc[i];
        }
        OUT* y = Y + row[i] * (unsigned long long)ldy + col[i];
        if (VEC) {
            if (n >= 16) {
                if constexpr (sizeof(OUT) == 2) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        reinterpret_cast<uint4*>(y)[k] =
                            make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                                       pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        reinterpret_cast<float4*>(y)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (k < n) y[k] = from_f32<OUT>(v[k]);
            }
        } else {                       // the warp's 512 values, 32 neighbours at a time
            const int lane = threadIdx.x & 31;
            OUT* mine = stage + threadIdx.x * 17;
#pragma unroll
            for (int k = 0; k < 16; ++k) mine[k] = from_f32<OUT>(v[k]);
            __syncwarp();
            const OUT* warp = stage + (threadIdx.x & ~31) * 17;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int owner = 2 * k + (lane >> 4), e = lane & 15;
                const unsigned long long at = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(y), owner);
                const int m = __shfl_sync(0xffffffffu, n, owner);
                if (e < m) reinterpret_cast<OUT*>(at)[e] = warp[owner * 17 + e];
            }
            __syncwarp();
        }
    }
}

bool aligned16p(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename IN, bool E5M2, bool VEC>
cudaError_t run_quantize(const void* X, long long rows, int cols, long long ldx, const Fp8View& out, void* copy,
                         cudaStream_t s) {
    const int nb = (cols + kFp8Block - 1) / kFp8Block, step = kThreads / 8,
              per = step * kBlocks<IN>;
    const unsigned long long blocks = (unsigned long long)rows * nb;
    const unsigned grid = (unsigned)((blocks + per - 1) / per);
    auto k = quantize_kernel<IN, E5M2, VEC, false>;
    if constexpr (std::is_same<IN, float>::value && VEC && !E5M2) {
        if (copy) k = quantize_kernel<IN, E5M2, VEC, true>;
    } else if (copy) {
        return cudaErrorNotSupported;
    }
    return launch_k(k, dim3(grid), dim3(kThreads), 0, s, (const IN*)X, blocks, cols, nb, step / nb, step % nb, ldx, out,
                    (__nv_bfloat16*)copy);
}

template <typename IN>
cudaError_t quantize_as(const void* X, long long rows, int cols, long long ldx, const Fp8View& out, void* copy,
                        cudaStream_t s) {
    const bool vec = aligned16p(X) && (ldx * sizeof(IN)) % 16 == 0;
    if (out.e5m2)
        return vec ? run_quantize<IN, true, true>(X, rows, cols, ldx, out, copy, s)
                   : run_quantize<IN, true, false>(X, rows, cols, ldx, out, copy, s);
    return vec ? run_quantize<IN, false, true>(X, rows, cols, ldx, out, copy, s)
               : run_quantize<IN, false, false>(X, rows, cols, ldx, out, copy, s);
}

template <typename OUT, bool E5M2>
cudaError_t dequantize_as(const Fp8View& in, long long rows, int cols, void* Y, long long ldy, cudaStream_t s) {
    const int nch = (cols + 15) / 16;
    const unsigned long long chunks = (unsigned long long)rows * nch;
    const unsigned grid = (unsigned)((chunks + kThreads * kUnroll - 1) / (kThreads * kUnroll));
    const bool vec = aligned16p(Y) && (ldy * sizeof(OUT)) % 16 == 0;
    return launch_k(vec ? dequantize_kernel<OUT, E5M2, true> : dequantize_kernel<OUT, E5M2, false>, dim3(grid),
                    dim3(kThreads), 0, s, in, chunks, cols, nch, kThreads / nch, kThreads % nch, (OUT*)Y, ldy);
}

}  // namespace

cudaError_t launch_fp8_quantize(bool f32, const void* X, long long rows, int cols, long long ldx, const Fp8View& out,
                                void* copy, cudaStream_t s) {
    RM_HOST_BOUNDS(rows >= 1 && cols >= 1 && ldx >= cols && fp8_on(X, f32 ? 4 : 2) && fp8_holds(out, cols));
    RM_HOST_BOUNDS(!copy || (cols % 16 == 0 && fp8_on(copy, 16)));
    return f32 ? quantize_as<float>(X, rows, cols, ldx, out, copy, s)
               : quantize_as<__nv_bfloat16>(X, rows, cols, ldx, out, copy, s);
}

cudaError_t launch_fp8_quantize_weight(bool f32, const void* W, int T, int K, int N, const Fp8View& out,
                                       cudaStream_t s) {
    RM_HOST_BOUNDS(T >= 1 && K >= 1 && N >= 1 && fp8_on(W, f32 ? 4 : 2) && fp8_holds(out, N) && !out.e5m2);
    const dim3 grid((N + kFp8Block - 1) / kFp8Block, (K + kFp8Block - 1) / kFp8Block, T);
    const bool vec = aligned16p(W) && (size_t)N * (f32 ? 4 : 2) % 16 == 0;
    if (f32)
        return launch_k(vec ? quantize_weight_kernel<float, true> : quantize_weight_kernel<float, false>, grid,
                        dim3(kThreads), 0, s, (const float*)W, K, N, out);
    return launch_k(vec ? quantize_weight_kernel<__nv_bfloat16, true> : quantize_weight_kernel<__nv_bfloat16, false>,
                    grid, dim3(kThreads), 0, s, (const __nv_bfloat16*)W, K, N, out);
}

cudaError_t launch_fp8_dequantize(const Fp8View& in, long long rows, int cols, void* Y, bool f32, long long ldy,
                                  cudaStream_t s) {
    RM_HOST_BOUNDS(rows >= 1 && cols >= 1 && ldy >= cols && fp8_on(Y, f32 ? 4 : 2) && fp8_holds(in, cols));
    if (f32)
        return in.e5m2 ? dequantize_as<float, true>(in, rows, cols, Y, ldy, s)
                       : dequantize_as<float, false>(in, rows, cols, Y, ldy, s);
    return in.e5m2 ? dequantize_as<__nv_bfloat16, true>(in, rows, cols, Y, ldy, s)
                   : dequantize_as<__nv_bfloat16, false>(in, rows, cols, Y, ldy, s);
}

}  // namespace rm
