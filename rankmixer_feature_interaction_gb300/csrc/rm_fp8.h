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

// For the launchers' checks in the debug build: rows that hold `cols` codes and their exponent bytes.
inline bool fp8_on(const void* p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }
inline bool fp8_holds(const Fp8View& v, int cols) {
    return fp8_on(v.codes, 16) && fp8_on(v.scales, 4) && v.ld >= cols && v.ld % 16 == 0 &&
           v.lds >= (cols + kFp8Block - 1) / kFp8Block && v.lds % 4 == 0;
}

// X [rows][ldx] (float, or bf16) -> out.  copy (nullable; of 16-byte aligned float
// rows to e4m3 only): the rows in bf16, [rows][cols] contiguous, cols a multiple of 16.
cudaError_t launch_fp8_quantize(bool f32, const void* X, long long rows, int cols, long long ldx, const Fp8View& out,
                                void* copy, cudaStream_t s);
cudaError_t launch_fp8_quantize_weight(bool f32, const void* W, int T, int K, int N, const Fp8View& out,
                                       cudaStream_t s);
cudaError_t launch_fp8_dequantize(const Fp8View& in, long long rows, int cols, void* Y, bool f32, long long ldy,
                                  cudaStream_t s);

// What the tensor-core kernels need of the current device: its SM count, the
// error word that bounded waits latch and their bound.
struct Fp8Device {
    int num_sms;
    int* err;
    unsigned long long timeout_ns;
};
// Of the current device, looked up once per device; RM_OK (0) or the call's status.
int fp8_device(Fp8Device* out);

// acc[b][t][n] = sum_k x[b][t][k] W[t][k][n] (trans: W[t][n][k]), then
//   FP8_OUT_*:  y = acc + bias (bias nullable)
//   FP8_GELU:   u = acc + bias; o0 = Q(Gelu(u)) and, where o1.codes is not null, o1 = Q(u)
//   FP8_DGELU:  dU = acc Gelu'(u) with u read from o1; o0 = Q(dU), y = dU in bf16 (the operand
//               of dW1: at most 2^-8 of each value, as large as a bf16 gradient's own rounding, where
//               Q(dU) would be off by up to 2^-4 and float32 halve that product's rate)
enum Fp8Epilogue { FP8_OUT_BF16, FP8_OUT_F32, FP8_GELU, FP8_DGELU };
struct Fp8Product {
    Fp8Epilogue epi;
    Fp8View x, w;
    bool trans;
    const float* bias;
    void* y;
    Fp8View o0, o1;
    int B, T, K, N;
    bool follows = false;       // launched right after another kernel of the same call (which waited for its
                                // own predecessor before this one could start): W is in memory already
};
// Up to this many samples the weights are streamed past all of them at once (launch_fp8_stream) instead of
// in tiles of 256 samples: at 64 samples T = 32, K = 1536, N = 6144 takes 54 us against 64, at 128 61 against
// 66.5; T = 8, K = 512, N = 2048 takes 3.5 and 4.1 us against 6.4 and 7.0.  (Closest for the
// training forward, at 72 samples of T = 32, D = 1536, F = 6144: 132 us against 133.)
// More samples go there too where that makes no more tiles than SMs: T = 8, K = 2048, N = 512, 250 samples (64
// tiles) 8.9 us against 10.1, T = 2, K = 256, N = 512, 1000 samples (64 tiles) 3.6 against 5.7; past one tile
// per SM it loses: T = 8, K = 2048, N = 512, 768 samples (192 tiles) 14.8 us against 11.0.
constexpr int kFp8StreamMaxB = 128;
// dU (FP8_DGELU) reads the kept u a byte at a time there and has no table of Gelu', so only up to 32 samples:
// the backward pass of T = 8, D = 512, F = 2048 takes 28.2 us at 1 sample and 30.3 at 32, against 33.2 and 33.9;
// T = 32, D = 1536, F = 6144 342 against 354 at 32, but 386 against 367 at 64.
constexpr int kFp8StreamMaxBdU = 32;
bool fp8_streams(const Fp8Product& p, const Fp8Device& dev);
cudaError_t launch_fp8_stream(const Fp8Product& p, const Fp8Device& dev, cudaStream_t s);
cudaError_t launch_fp8_product(const Fp8Product& p, const Fp8Device& dev, cudaStream_t s);

// dW[t][k][n] = sum_b x[b][t][k] dY[b][t][n] and, where db is not null, db[t][n] =
// sum_b dY[b][t][n], both float or both bf16; dY bf16 [B][T][N].
cudaError_t launch_fp8_wgrad(const Fp8View& x, const void* dY, void* dW, void* db, bool f32, int B, int T, int K, int N,
                             const Fp8Device& dev, cudaStream_t s);

}  // namespace rm
