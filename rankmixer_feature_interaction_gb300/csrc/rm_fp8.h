// Internal launcher interface of the 8-bit operators (include/rankmixer.h,
// "8-bit operands and checkpoints").  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rm_internal.h"

namespace rm {

constexpr int kFp8Block = 128;      // values that share one exponent byte

// Rows of codes with their exponent bytes; e5m2 tells the format (else e4m3).
struct Fp8View {
    uint8_t* codes;
    uint8_t* scales;
    long long ld, lds;
    bool e5m2;
};

// X [rows][ldx] (float, or bf16) -> out.  copy (nullable): the rows in bf16,
// [rows][cols] contiguous, cols a multiple of 8.
cudaError_t launch_fp8_quantize(bool f32, const void* X, long long rows, int cols, long long ldx, const Fp8View& out,
                                void* copy, cudaStream_t s);
cudaError_t launch_fp8_quantize_weight(bool f32, const void* W, int T, int K, int N, const Fp8View& out,
                                       cudaStream_t s);
cudaError_t launch_fp8_dequantize(const Fp8View& in, long long rows, int cols, void* Y, bool f32, long long ldy,
                                  cudaStream_t s);

// out[t][n] = sum over b of Y[b][t][n] (bf16, [B][T][N], N a multiple of 8), of
// float or bf16, in a fixed order.
cudaError_t launch_fp8_colsum(const void* Y, void* out, bool out_f32, int B, int T, int N, cudaStream_t s);

// Y[b][t][n] = sum_k x[b][t][k] W[t][k][n] (trans: W[t][n][k]) + bias[t][n].
cudaError_t launch_fp8_matmul(const Fp8View& x, const Fp8View& w, bool trans, const float* bias, void* Y, bool y_f32,
                              int B, int T, int K, int N, cudaStream_t s);

// dW[t][k][n] = sum_b x[b][t][k] dY[b][t][n], dY bf16 [B][T][N].
cudaError_t launch_fp8_wgrad(const Fp8View& x, const void* dY, void* dW, bool w_f32, int B, int T, int K, int N,
                             cudaStream_t s);

// From u = x W1 + b1 [rows][cols] in float: a = Q(Gelu(u)) and, where u8.codes
// is not null, u8 = Q(u).
cudaError_t launch_fp8_gelu(const float* u, long long rows, int cols, const Fp8View& a, const Fp8View& u8,
                            cudaStream_t s);

// From dA [rows][cols] in float and the kept u8: dU = dA Gelu'(u) as d8 = Q(dU) and in bf16.
cudaError_t launch_fp8_dgelu(const float* dA, long long rows, int cols, const Fp8View& u8, const Fp8View& d8, void* dU,
                             cudaStream_t s);

}  // namespace rm
