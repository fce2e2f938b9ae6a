// Products of 4-bit operands, in the simplest form: a thread per column, the rows of a
// tile one after another, codes and scales read where they lie.
#include "rm_fp4.cuh"
#include "rm_fp8.cuh"

namespace rm {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float scale_of(uint32_t E) { return fp8_scale(E); }

template <int EPI>
__global__ void __launch_bounds__(kThreads)
product_kernel(Fp4Product p, long long n_rows) {
    pdl_wait();
    pdl_launch_next();
    const int n = blockIdx.x * kThreads + threadIdx.x, nb = (p.K + kFp4Block - 1) / kFp4Block;
    const bool live = n < p.N;
    const long long tiles_n = (p.N + kFp4TileRows - 1) / kFp4TileRows;
    long long units = p.tiles ? p.tiles[0].x : (long long)p.B * p.G;
    for (long long u = blockIdx.y; u < units; u += gridDim.y) {
        int g, rows = 1;
        long long row0;
        if (p.tiles) {
            const int4 t = p.tiles[1 + u];
            g = t.x, row0 = t.y, rows = t.z;
        } else {
            g = (int)(u % p.G), row0 = u;
        }
        for (int i = 0; i < rows && row0 + i < n_rows; ++i) {
            const long long row = row0 + i;
            float acc = 0.f;
            if (live)
                for (int b = 0; b < nb; ++b) {
                    const uint4 xc = *reinterpret_cast<const uint4*>(p.x.codes + row * p.x.ld + 16 * b);
                    const uint4 wc = *reinterpret_cast<const uint4*>(p.w.codes + ((long long)g * p.N + n) * p.w.ld + 16 * b);
                    const uint32_t* xw = &xc.x;
                    const uint32_t* ww = &wc.x;
                    const uint8_t ws = p.w.scales[(((long long)g * tiles_n + n / 128) * p.w.lds + b / 4) * 512 + 16 * (n % 32) +
                                                  4 * (n % 128 / 32) + b % 4];
                    const float s = scale_of(p.x.scales[row * p.x.lds + b]) * scale_of(ws);
                    float sum = 0.f;
                    for (int q = 0; q < 4; ++q) {
                        float a[8], w[8];
                        fp4_unpack8(xw[q], a);
                        fp4_unpack8(ww[q], w);
                        for (int k = 0; k < 8; ++k) sum = fmaf(a[k], w[k], sum);
                    }
                    acc = fmaf(s, sum, acc);
                }
            if (p.bias && live) acc += p.bias[(long long)g * p.N + n];
            if (EPI == FP4_GELU) {
                const float a = live ? fp8_gelu(acc) : 0.f;
                const uint32_t E = fp4_exponent(__reduce_max_sync(0xffffffffu, fp4_abs_bits(a)));
                float v[8];
                for (int k = 0; k < 8; ++k) v[k] = __shfl_sync(0xffffffffu, a, (threadIdx.x & 24) + k) * fp4_inv_scale(E);
                const uint32_t c = fp4_pack8(v);
                if (live && (threadIdx.x & 7) == 0) *reinterpret_cast<uint32_t*>(p.o.codes + row * p.o.ld + n / 2) = c;
                if (live && (threadIdx.x & 31) == 0) p.o.scales[row * p.o.lds + n / 32] = (uint8_t)E;
            } else if (live) {
                if (EPI == FP4_OUT_F32)
                    static_cast<float*>(p.y)[row * p.N + n] = acc;
                else
                    static_cast<__nv_bfloat16*>(p.y)[row * p.N + n] = __float2bfloat16_rn(acc);
            }
        }
    }
}

}  // namespace

cudaError_t launch_fp4_product(const Fp4Product& p, const Fp8Device& dev, cudaStream_t s) {
    const long long rows = p.tiles ? p.n : (long long)p.B * p.G;
    const dim3 grid((unsigned)((p.N + kThreads - 1) / kThreads), (unsigned)(rows < 4096 ? (rows ? rows : 1) : 4096));
    switch (p.epi) {
        case FP4_OUT_BF16: return launch_k(product_kernel<FP4_OUT_BF16>, grid, dim3(kThreads), 0, s, p, rows);
        case FP4_OUT_F32: return launch_k(product_kernel<FP4_OUT_F32>, grid, dim3(kThreads), 0, s, p, rows);
        case FP4_GELU: return launch_k(product_kernel<FP4_GELU>, grid, dim3(kThreads), 0, s, p, rows);
    }
    return cudaErrorNotSupported;
}

}  // namespace rm
