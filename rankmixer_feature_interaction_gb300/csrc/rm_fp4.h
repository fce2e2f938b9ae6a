// Internal launcher interface of the 4-bit operators and of the experts' rows
// (include/rankmixer.h, "4-bit operands" and "Rows by expert").  Not part of the
// public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rm_fp8.h"
#include "rm_internal.h"

namespace rm {

constexpr int kFp4Block = 32;       // values that share one exponent byte
constexpr int kFp4TileRows = 128;   // rows of a weight whose exponent bytes lie together
constexpr int kFp4KBlock = 256;     // values of K per step of the products (128 bytes of codes)

// Rows of codes (two a byte) with their exponent bytes.  Activations: row r's bytes
// at scales + r lds.  Weights: 512 bytes per 128 rows and 128 values of K, lds of
// them per 128 rows (fp4_weight_quads of K).
struct Fp4View {
    uint8_t* codes;
    uint8_t* scales;
    long long ld, lds;
};
inline long long fp4_blocks(long long cols) { return (cols + kFp4Block - 1) / kFp4Block; }
inline long long fp4_weight_quads(long long K) { return 2 * ((K + kFp4KBlock - 1) / kFp4KBlock); }
inline bool fp4_holds(const Fp4View& v, long long cols) {
    return fp8_on(v.codes, 16) && fp8_on(v.scales, 16) && v.ld % 16 == 0 && v.ld >= 16 * fp4_blocks(cols) &&
           v.lds % 16 == 0 && v.lds >= fp4_blocks(cols);
}

// A sort of the open (t, e, b): include/rankmixer.h, rm_expert_rows.  tiles[0].x is
// the number of tiles, tiles[1 + i] = {group, first row, rows (at most kExpertTile), 0}.
constexpr int kExpertTile = 256;
struct ExpertRows {
    int* offsets;
    int* source;
    int* slot;
    int4* tiles;
    int B, T, E;
};

cudaError_t launch_fp4_quantize(bool f32, const void* X, long long rows, int cols, long long ldx, const Fp4View& out,
                                cudaStream_t s);
cudaError_t launch_fp4_dequantize(const Fp4View& in, long long rows, int cols, void* Y, bool f32, long long ldy,
                                  cudaStream_t s);
// W [G][K][N] -> rows (g, n) along K.
cudaError_t launch_fp4_quantize_weight(bool f32, const void* W, int G, int K, int N, const Fp4View& out, cudaStream_t s);

// Workspace of the sort, in ints.
long long expert_sort_work(int B, int T, int E);
cudaError_t launch_expert_sort(const float* G, const ExpertRows& r, int* work, cudaStream_t s);
// Xs[slot] = X[b][t] for every open slot below n; or the same row in 4 bits.
cudaError_t launch_expert_gather(const void* X, bool f32, const ExpertRows& r, void* Xs, long long n, int D,
                                 cudaStream_t s);
cudaError_t launch_fp4_expert_gather(const void* X, bool f32, const ExpertRows& r, const Fp4View& out, long long n, int D,
                                     cudaStream_t s);
// V[b][t] = sum over the open e of G[b][t][e] Y[slot] (G null: of Y[slot]).
cudaError_t launch_expert_combine(const void* Y, bool y_f32, const ExpertRows& r, const float* G, void* V, bool v_f32,
                                  long long n, int D, cudaStream_t s);
// dY[slot] = G dV[b][t], dG = Y[slot] . dV[b][t] (0 where closed).
cudaError_t launch_expert_combine_backward(const void* dV, const void* Y, bool f32, const ExpertRows& r, const float* G,
                                           void* dY, float* dG, long long n, int D, cudaStream_t s);

// y[row][n] = sum_k x[row][k] W[g][n][k] + bias[g][n] over the rows of group g; FP4_GELU: o = Q(Gelu(y)).
// Per token (tiles null): groups are the T tokens, row (b, t) at b T + t.  By expert: the sorted rows, group t E + e.
enum Fp4Epilogue { FP4_OUT_BF16, FP4_OUT_F32, FP4_GELU };
struct Fp4Product {
    Fp4Epilogue epi;
    Fp4View x, w;
    const float* bias;
    void* y;
    Fp4View o;
    const int4* tiles;
    long long n;                // rows of x that exist in memory (by expert)
    int B, G, K, N;             // B: rows of a group at most; G: groups
    bool follows = false;       // as in Fp8Product
};
cudaError_t launch_fp4_product(const Fp4Product& p, const Fp8Device& dev, cudaStream_t s);

}  // namespace rm
