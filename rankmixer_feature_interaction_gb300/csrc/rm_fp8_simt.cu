// The weight-gradient product of the 8-bit operators on the CUDA cores, 64 x 64 tiles with
// operands restored to float32 in shared memory.
#include "rm_common.cuh"
#include "rm_fp8.cuh"

namespace rm {
namespace {

constexpr int TILE = 64, KSTEP = 16;

__device__ __forceinline__ float code_value(uint8_t c, bool e5m2) {
    return e5m2 ? fp8_unpack2<true>(c).x : fp8_unpack2<false>(c).x;
}

struct RowsX {      // A(m = b, k) = x[b][t][k]
    Fp8View x;
    int T;
    __device__ float operator()(int t, int b, int k) const {
        const size_t r = (size_t)b * T + t;
        return code_value(x.codes[r * x.ld + k], x.e5m2) * fp8_scale(x.scales[r * x.lds + k / kFp8Block]);
    }
};
struct ColsX {      // A(m = k, b) = x[b][t][k]
    RowsX x;
    __device__ float operator()(int t, int k, int b) const { return x(t, b, k); }
};
struct RowsY {      // B(b, n) = dY[b][t][n]
    const __nv_bfloat16* y;
    int T, N;
    __device__ float operator()(int t, int b, int n) const { return to_f32(y[((size_t)b * T + t) * N + n]); }
};
template <typename OUT>
struct ToW {        // dW[t][k][n]
    OUT* w;
    int K, N;
    __device__ void operator()(int t, int k, int n, float v) const { w[((size_t)t * K + k) * N + n] = from_f32<OUT>(v); }
};

template <class A, class B, class C>
__global__ void __launch_bounds__(256) product_kernel(A a, B b, C c, int M, int N, int K) {
    __shared__ float sa[KSTEP][TILE + 1], sb[KSTEP][TILE + 1];
    const int t = blockIdx.z, m0 = blockIdx.y * TILE, n0 = blockIdx.x * TILE;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += KSTEP) {
        for (int i = threadIdx.x; i < TILE * KSTEP; i += 256) {
            const int r = i / KSTEP, k = i % KSTEP;
            sa[k][r] = m0 + r < M && k0 + k < K ? a(t, m0 + r, k0 + k) : 0.f;
            const int kk = i / TILE, n = i % TILE;
            sb[kk][n] = n0 + n < N && k0 + kk < K ? b(t, k0 + kk, n0 + n) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KSTEP; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < M && n < N) c(t, m, n, acc[i][j]);
        }
}

template <class A, class B, class C>
cudaError_t run(const A& a, const B& b, const C& c, int T, int M, int N, int K, cudaStream_t s) {
    product_kernel<<<dim3((N + TILE - 1) / TILE, (M + TILE - 1) / TILE, T), 256, 0, s>>>(a, b, c, M, N, K);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_wgrad(const Fp8View& x, const void* dY, void* dW, bool w_f32, int B, int T, int K, int N,
                             cudaStream_t s) {
    const ColsX a{RowsX{x, T}};
    const RowsY b{(const __nv_bfloat16*)dY, T, N};
    if (w_f32) return run(a, b, ToW<float>{(float*)dW, K, N}, T, K, N, B, s);
    return run(a, b, ToW<__nv_bfloat16>{(__nv_bfloat16*)dW, K, N}, T, K, N, B, s);
}

}  // namespace rm
