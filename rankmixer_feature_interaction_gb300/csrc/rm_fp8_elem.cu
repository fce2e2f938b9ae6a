// Elementwise kernels of the 8-bit operators: saving rows and weights in 8 bits,
// and restoring rows.
//
// Saving reads every value once and writes one byte for it; 16 lanes own one
// block of 128 values (8 each: one or two 16-byte loads), agree on its largest
// magnitude with four shuffles and write 8 bytes of codes each.  Four blocks
// per half warp are loaded before the first is used.
#include "rm_common.cuh"
#include "rm_fp8.cuh"

namespace rm {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

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

// Largest of 16 lanes, for all of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// One block of a row: 8 values per lane of a half warp (n of them inside the row).
template <bool E5M2>
__device__ __forceinline__ void save_block(const float (&v)[8], int n, int l16, uint8_t* codes, uint8_t* scale,
                                           int room) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, fp8_finite_bits(v[i]));
    const uint32_t E = fp8_exponent<E5M2>(max16(m));
    const float s = fp8_inv_scale(E);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fp8_poison(v[i]) * s;
    if (room >= 8) {        // code rows are padded to 16 bytes, so a lane's 8 bytes fit or are not there at all
        const uint2 w = make_uint2(fp8_pack4<E5M2>(q[0], q[1], q[2], q[3]), fp8_pack4<E5M2>(q[4], q[5], q[6], q[7]));
        *reinterpret_cast<uint2*>(codes) = w;
    }
    if (l16 == 0 && n > 0) *scale = (uint8_t)E;
}

template <typename IN, bool E5M2, bool VEC, bool COPY>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const IN* __restrict__ X, unsigned long long blocks, int cols, int nb, long long ldx, Fp8View out,
                __nv_bfloat16* __restrict__ copy) {
    pdl_wait();
    pdl_launch_next();
    const int l16 = threadIdx.x & 15;
    const unsigned long long base = (unsigned long long)blockIdx.x * (kThreads / 16 * kUnroll) + (threadIdx.x >> 4);
    float v[kUnroll][8];
    unsigned long long row[kUnroll];
    int col[kUnroll], left[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const unsigned long long id = base + (unsigned long long)i * (kThreads / 16);
        unsigned long long r = 0;
        int j = 0;
        left[i] = 0;
        if (id < blocks) {
            if (blocks <= 0xffffffffull) {
                r = (uint32_t)id / (uint32_t)nb;
                j = (int)((uint32_t)id - (uint32_t)r * (uint32_t)nb);
            } else {
                r = id / (unsigned)nb;
                j = (int)(id - r * (unsigned)nb);
            }
            left[i] = cols - (j * kFp8Block + 8 * l16);
        }
        row[i] = r;
        col[i] = j * kFp8Block + 8 * l16;
        load8<IN, VEC>(X + r * (unsigned long long)ldx + col[i], left[i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const bool here = base + (unsigned long long)i * (kThreads / 16) < blocks;
        const int room = here ? (cols + 15) / 16 * 16 - col[i] : 0;
        save_block<E5M2>(v[i], here ? cols - (col[i] - 8 * l16) : 0, l16,
                         out.codes + row[i] * (unsigned long long)out.ld + col[i],
                         out.scales + row[i] * (unsigned long long)out.lds + col[i] / kFp8Block, room);
        if (COPY && left[i] >= 8) {
            uint4 w;
            w.x = pack_bf16x2(v[i][0], v[i][1]);
            w.y = pack_bf16x2(v[i][2], v[i][3]);
            w.z = pack_bf16x2(v[i][4], v[i][5]);
            w.w = pack_bf16x2(v[i][6], v[i][7]);
            *reinterpret_cast<uint4*>(copy + row[i] * (unsigned long long)cols + col[i]) = w;
        }
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
dequantize_kernel(Fp8View in, unsigned long long chunks, int cols, int nch, OUT* __restrict__ Y, long long ldy) {
    pdl_wait();
    pdl_launch_next();
    // one thread per 16 codes; four chunks in flight
    unsigned long long base = (unsigned long long)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint4 w[kUnroll];
    float sc[kUnroll];
    unsigned long long row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const unsigned long long id = base + (unsigned long long)i * kThreads;
        row[i] = 0;
        col[i] = cols;
        if (id < chunks) {
            unsigned long long r;
            if (chunks <= 0xffffffffull)
                r = (uint32_t)id / (uint32_t)nch;
            else
                r = id / (unsigned)nch;
            row[i] = r;
            col[i] = (int)(id - r * (unsigned)nch) * 16;
            w[i] = *reinterpret_cast<const uint4*>(in.codes + r * (unsigned long long)in.ld + col[i]);
            sc[i] = fp8_scale(in.scales[r * (unsigned long long)in.lds + col[i] / kFp8Block]);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int n = cols - col[i];
        if (n <= 0) continue;
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = fp8_unpack2<E5M2>(u[j >> 1] >> (16 * (j & 1)));
            v[2 * j] = f.x * sc[i];
            v[2 * j + 1] = f.y * sc[i];
        }
        OUT* y = Y + row[i] * (unsigned long long)ldy + col[i];
        if (VEC && n >= 16) {
            if constexpr (sizeof(OUT) == 2) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    reinterpret_cast<uint4*>(y)[j] =
                        make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                   pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    reinterpret_cast<float4*>(y)[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < n) y[j] = from_f32<OUT>(v[j]);
        }
    }
}

bool aligned16p(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename IN, bool E5M2, bool VEC>
cudaError_t run_quantize(const void* X, long long rows, int cols, long long ldx, const Fp8View& out, void* copy,
                         cudaStream_t s) {
    const int nb = (cols + kFp8Block - 1) / kFp8Block;
    const unsigned long long blocks = (unsigned long long)rows * nb;
    const unsigned grid = (unsigned)((blocks + kThreads / 16 * kUnroll - 1) / (kThreads / 16 * kUnroll));
    return launch_k(copy ? quantize_kernel<IN, E5M2, VEC, true> : quantize_kernel<IN, E5M2, VEC, false>, dim3(grid),
                    dim3(kThreads), 0, s, (const IN*)X, blocks, cols, nb, ldx, out, (__nv_bfloat16*)copy);
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
                    dim3(kThreads), 0, s, in, chunks, cols, nch, (OUT*)Y, ldy);
}

}  // namespace

cudaError_t launch_fp8_quantize(bool f32, const void* X, long long rows, int cols, long long ldx, const Fp8View& out,
                                void* copy, cudaStream_t s) {
    return f32 ? quantize_as<float>(X, rows, cols, ldx, out, copy, s)
               : quantize_as<__nv_bfloat16>(X, rows, cols, ldx, out, copy, s);
}

cudaError_t launch_fp8_quantize_weight(bool f32, const void* W, int T, int K, int N, const Fp8View& out,
                                       cudaStream_t s) {
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
    if (f32)
        return in.e5m2 ? dequantize_as<float, true>(in, rows, cols, Y, ldy, s)
                       : dequantize_as<float, false>(in, rows, cols, Y, ldy, s);
    return in.e5m2 ? dequantize_as<__nv_bfloat16, true>(in, rows, cols, Y, ldy, s)
                   : dequantize_as<__nv_bfloat16, false>(in, rows, cols, Y, ldy, s);
}

}  // namespace rm
