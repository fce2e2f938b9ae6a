// Elementwise kernels of the 4-bit operators: rows and weights to 4 bits, rows back.
//
// Rows: two neighbouring lanes own a block of 32 values, 16 each (32 bytes of bf16),
// agree on its largest magnitude with one shuffle and write eight bytes of codes each,
// so a warp reads a kilobyte of bf16 in a row and writes 256 bytes.  What a thread has
// loaded stays as it came until it is rounded: few registers, so many loads under way.
// Measured, 65,536 rows of 6144 in bf16: to 4 bits 147 us (6.9 TB/s; 326 with eight values
// a lane, unpacked at once), back 154 us (6.6 TB/s): bound by memory, 2.53 bytes a value.
// Rows that are not 16-byte aligned go by 16-byte pieces of memory too, those around the
// values, which are then shifted into place: 126,840 bf16 rows of 1547 to 4 bits 95 us
// (1552 columns, aligned: 79), back 119 us (80).  An element at a time, their order
// changed in shared memory, they took 262 and 160 us, and 47,720 rows of 33 15.7 us (4).
#include "rm_fp4.cuh"

namespace rm {
namespace {

constexpr int kThreads = 256;

// Row and piece of a running number (pieces of a row: n).
__device__ __forceinline__ void split(unsigned long long id, bool small, unsigned n, unsigned long long& row, int& j) {
    if (small) {
        const uint32_t r = (uint32_t)id / n;
        row = r, j = (int)((uint32_t)id - r * n);
    } else {
        row = id / n, j = (int)(id - row * n);
    }
}

// Row and piece of the running number that is `step` (dq rows and dr pieces) further.
__device__ __forceinline__ void advance(unsigned long long& row, int& j, int dq, int dr, int n) {
    row += dq, j += dr;
    if (j >= n) j -= n, ++row;
}

template <typename IN>
constexpr int kInFlight = sizeof(IN) == 2 ? 4 : 2;      // pieces of 16 values per thread

template <typename IN>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const IN* __restrict__ X, unsigned long long pieces, int cols, int nb, int dq, int dr, long long ldx,
                Fp4View out) {
    constexpr int UNROLL = kInFlight<IN>;
    pdl_wait();
    pdl_launch_next();
    const unsigned long long base = (unsigned long long)blockIdx.x * (kThreads * UNROLL) + threadIdx.x;
    unsigned long long row;
    int j;
    split(base, pieces <= 0xffffffffull, 2u * nb, row, j);
    Fp4Raw16<IN> v[UNROLL];
    unsigned long long at = row;
    int k = j;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const bool there = base + (unsigned long long)u * kThreads < pieces;
        v[u].template load<true>(X + at * ldx + 16 * k, there ? cols - 16 * k : 0);
        advance(at, k, dq, dr, 2 * nb);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        uint32_t E;
        const uint2 c = v[u].round(E);
        if (base + (unsigned long long)u * kThreads < pieces) {
            *reinterpret_cast<uint2*>(out.codes + row * out.ld + 8 * j) = c;
            if ((j & 1) == 0) out.scales[row * out.lds + (j >> 1)] = (uint8_t)E;
        }
        advance(row, j, dq, dr, 2 * nb);
    }
}

// Other rows: a lane reads the 16-byte pieces around its values and shifts them, one
// block half a thread (four in flight took registers: 110 us where one took 103); size:
// X's values from its first to its last.
template <typename IN>
__global__ void __launch_bounds__(kThreads)
quantize_odd_kernel(const IN* __restrict__ X, unsigned long long pieces, int cols, int nb, long long ldx,
                    unsigned long long size, Fp4View out) {
    pdl_wait();
    pdl_launch_next();
    const unsigned long long id = (unsigned long long)blockIdx.x * kThreads + threadIdx.x;
    const bool there = id < pieces;
    unsigned long long row;
    int j;
    split(there ? id : pieces - 1, pieces <= 0xffffffffull, 2u * nb, row, j);
    Fp4Raw16<IN> v;
    v.load_any(X, row * ldx + 16 * j, cols - 16 * j, size);
    uint32_t E;
    const uint2 c = v.round(E);
    if (there) {
        *reinterpret_cast<uint2*>(out.codes + row * out.ld + 8 * j) = c;
        if ((j & 1) == 0) out.scales[row * out.lds + (j >> 1)] = (uint8_t)E;
    }
}

// 2^(E - 127); 0 stands for 2^-127, 255 for NaN
__device__ __forceinline__ float fp4_scale(uint32_t E) {
    return E == 0u ? __uint_as_float(0x00400000u) : E == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(E << 23);
}

// Eight values to a 16-byte boundary.
template <typename OUT>
__device__ __forceinline__ void store8(OUT* y, const float (&v)[8]) {
    if constexpr (sizeof(OUT) == 2) {
        __stcs(reinterpret_cast<uint4*>(y), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    } else {
        __stcs(reinterpret_cast<float4*>(y), make_float4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<float4*>(y) + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
}

template <typename OUT>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(Fp4View in, unsigned long long pieces, int cols, int nb, OUT* __restrict__ Y, long long ldy) {
    constexpr int UNROLL = 4;
    pdl_wait();
    pdl_launch_next();
    const unsigned long long base = (unsigned long long)blockIdx.x * (kThreads * UNROLL) + threadIdx.x;
    const bool small = pieces <= 0xffffffffull;
    uint32_t c[UNROLL], E[UNROLL];
    unsigned long long row[UNROLL];
    int j[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const unsigned long long id = base + (unsigned long long)u * kThreads;
        split(id < pieces ? id : pieces - 1, small, 4u * nb, row[u], j[u]);
        c[u] = *reinterpret_cast<const uint32_t*>(in.codes + row[u] * in.ld + 4 * j[u]);
        E[u] = in.scales[row[u] * in.lds + (j[u] >> 2)];
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (base + (unsigned long long)u * kThreads >= pieces) return;
        float v[8];
        fp4_unpack8(c[u], v);
        const float s = fp4_scale(E[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= s;
        OUT* y = Y + row[u] * ldy + 8 * j[u];
        const int n = cols - 8 * j[u];
        if (n >= 8) {
            store8(y, v);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) y[i] = from_f32<OUT>(v[i]);
        }
    }
}

// Other rows: a lane writes eight values from a 16-byte boundary of the output on, of
// which a row's first and last piece may hold fewer; per_row: the most pieces of a row.
template <typename OUT>
__global__ void __launch_bounds__(kThreads)
dequantize_odd_kernel(Fp4View in, unsigned long long pieces, int cols, int nb, int per_row, OUT* __restrict__ Y,
                      long long ldy) {
    constexpr int UNROLL = 4;
    pdl_wait();
    pdl_launch_next();
    const unsigned long long base = (unsigned long long)blockIdx.x * (kThreads * UNROLL) + threadIdx.x;
    const bool small = pieces <= 0xffffffffull;
    uint32_t w[UNROLL][2], E[UNROLL][2];
    unsigned long long row[UNROLL];
    int j[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        const unsigned long long id = base + (unsigned long long)u * kThreads;
        split(id < pieces ? id : pieces - 1, small, per_row, row[u], j[u]);
        // words j - 1 and j of the row's codes, where it has them
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = j[u] - 1 + i;
            const bool is = k >= 0 && k < 4 * nb;
            w[u][i] = is ? *reinterpret_cast<const uint32_t*>(in.codes + row[u] * in.ld + 4 * k) : 0u;
            E[u][i] = is ? in.scales[row[u] * in.lds + (k >> 2)] : 0u;
        }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (base + (unsigned long long)u * kThreads >= pieces) return;
        OUT* y = Y + row[u] * ldy;
        const int o = (int)(reinterpret_cast<uintptr_t>(y) % 16 / sizeof(OUT));     // values before the row in its first piece
        const float s0 = fp4_scale(E[u][0]), s1 = fp4_scale(E[u][1]);
        float v[8];
        fp4_unpack8(__funnelshift_rc(w[u][0], w[u][1], 4 * (8 - o)), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= i < o ? s0 : s1;
        const uint32_t c = 8u * j[u] - o;           // before the row: a column past every other
        if (cols >= 8 && c <= (uint32_t)cols - 8u) {
            store8(y + c, v);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i)
                if (c + i < (uint32_t)cols) y[c + i] = from_f32<OUT>(v[i]);
        }
    }
}

// Weights [G][K][N] to rows along K: a thread owns 128 values of K of two neighbouring
// columns (of one where rows of W are not aligned to pairs), 32 at a time, so that a warp
// reads 128 bytes of a row of bf16; it writes 16 bytes of codes a block and the word of
// four exponent bytes where the products read it.  Columns past N and blocks past K get
// exponent bytes of 127.  302 M weights from bf16 152 us (5.0 TB/s; one column a thread
// 322), from float32 203 (6.7 TB/s).
constexpr int kWeightThreads = 128;
template <typename IN, int COLS>
struct WeightBlock {
    uint32_t w[sizeof(IN) == 2 ? 32 : 32 * COLS];       // bf16: the columns side by side
    __device__ __forceinline__ void load(const IN* p, size_t N, int left) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if constexpr (sizeof(IN) == 2) {
                w[i] = 0;
                if (i < left)
                    w[i] = COLS == 2 ? *reinterpret_cast<const uint32_t*>(p + i * N) : __bfloat16_as_ushort(p[i * N]);
            } else if constexpr (COLS == 2) {
                const uint2 v = i < left ? *reinterpret_cast<const uint2*>(p + i * N) : make_uint2(0, 0);
                w[2 * i] = v.x, w[2 * i + 1] = v.y;
            } else {
                w[i] = i < left ? __float_as_uint(p[i * N]) : 0u;
            }
        }
    }
    __device__ __forceinline__ float get(int i, int c) const {
        if constexpr (sizeof(IN) == 2) return __uint_as_float(c ? w[i] & 0xffff0000u : w[i] << 16);
        return __uint_as_float(w[COLS * i + c]);
    }
    // 16 bytes of codes of column c; returns the exponent byte
    __device__ __forceinline__ uint32_t save(int c, uint8_t* codes) const {
        uint32_t m = 0, q[4];
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, fp4_abs_bits(get(i, c)));
        const uint32_t E = fp4_exponent(m);
        const float s = fp4_inv_scale(E);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = get(8 * i + k, c) * s;
            q[i] = fp4_pack8(v);
        }
        *reinterpret_cast<uint4*>(codes) = make_uint4(q[0], q[1], q[2], q[3]);
        return E;
    }
};
template <typename IN, int COLS>
__global__ void __launch_bounds__(kWeightThreads)
quantize_weight_kernel(const IN* __restrict__ W, int K, int N, int nb, Fp4View out) {
    constexpr int PER = kFp4TileRows / COLS;            // threads of a tile and quad
    pdl_wait();
    pdl_launch_next();
    const int tile = blockIdx.x, g = blockIdx.z, r = COLS * (threadIdx.x % PER), n = tile * kFp4TileRows + r;
    const long long tiles = (N + kFp4TileRows - 1) / kFp4TileRows;
    for (long long q = blockIdx.y * COLS + threadIdx.x / PER; q < out.lds; q += (long long)gridDim.y * COLS) {
        uint32_t word[COLS] = {};
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            const int b = (int)(4 * q) + c, k0 = kFp4Block * b;
            uint32_t E[COLS];
#pragma unroll
            for (int i = 0; i < COLS; ++i) E[i] = 127;
            if (n < N && b < nb) {                      // COLS divides N
                WeightBlock<IN, COLS> v;
                v.load(W + ((size_t)g * K + k0) * N + n, N, K - k0);
#pragma unroll
                for (int i = 0; i < COLS; ++i) E[i] = v.save(i, out.codes + ((size_t)g * N + n + i) * out.ld + 16 * (size_t)b);
            }
#pragma unroll
            for (int i = 0; i < COLS; ++i) word[i] |= E[i] << (8 * c);
        }
        uint8_t* at = out.scales + (((size_t)g * tiles + tile) * out.lds + q) * 512;
#pragma unroll
        for (int i = 0; i < COLS; ++i)
            *reinterpret_cast<uint32_t*>(at + 16 * ((r + i) & 31) + 4 * ((r + i) >> 5)) = word[i];
    }
}

bool rows_aligned(const void* p, long long ld, int esz) { return fp8_on(p, 16) && ld * esz % 16 == 0; }

template <typename IN>
cudaError_t quantize(const IN* X, long long rows, int cols, long long ldx, const Fp4View& out, cudaStream_t s) {
    const int nb = (int)fp4_blocks(cols);
    const bool aligned = rows_aligned(X, ldx, sizeof(IN));
    const int per = aligned ? kThreads * kInFlight<IN> : kThreads;
    const unsigned long long pieces = 2ull * rows * nb, grid = (pieces + per - 1) / per;
    if (grid > 0x7fffffffull) return cudaErrorNotSupported;
    if (aligned)
        return launch_k(quantize_kernel<IN>, dim3((unsigned)grid), dim3(kThreads), 0, s, X, pieces, cols, nb,
                        kThreads / (2 * nb), kThreads % (2 * nb), ldx, out);
    return launch_k(quantize_odd_kernel<IN>, dim3((unsigned)grid), dim3(kThreads), 0, s, X, pieces, cols, nb, ldx,
                    (unsigned long long)(rows - 1) * ldx + cols, out);
}

template <typename OUT>
cudaError_t dequantize(const Fp4View& in, long long rows, int cols, OUT* Y, long long ldy, cudaStream_t s) {
    const int nb = (int)fp4_blocks(cols);
    if (rows_aligned(Y, ldy, sizeof(OUT))) {
        const unsigned long long pieces = 4ull * rows * nb, grid = (pieces + 4 * kThreads - 1) / (4 * kThreads);
        if (grid > 0x7fffffffull) return cudaErrorNotSupported;
        return launch_k(dequantize_kernel<OUT>, dim3((unsigned)grid), dim3(kThreads), 0, s, in, pieces, cols, nb, Y, ldy);
    }
    const int per_row = (int)((cols + 16 / (long long)sizeof(OUT) - 1 + 7) / 8);
    const unsigned long long pieces = (unsigned long long)rows * per_row, grid = (pieces + 4 * kThreads - 1) / (4 * kThreads);
    if (grid > 0x7fffffffull) return cudaErrorNotSupported;
    return launch_k(dequantize_odd_kernel<OUT>, dim3((unsigned)grid), dim3(kThreads), 0, s, in, pieces, cols, nb, per_row, Y,
                    ldy);
}

template <typename IN>
cudaError_t quantize_weight(const IN* W, int G, int K, int N, const Fp4View& out, cudaStream_t s) {
    const bool pairs = N % 2 == 0 && fp8_on(W, 2 * sizeof(IN));
    const long long quads = pairs ? out.lds / 2 : out.lds;       // (lds is even)
    const dim3 grid((unsigned)((N + kFp4TileRows - 1) / kFp4TileRows), (unsigned)(quads < 65535 ? quads : 65535), (unsigned)G);
    return launch_k(pairs ? quantize_weight_kernel<IN, 2> : quantize_weight_kernel<IN, 1>, grid, dim3(kWeightThreads), 0, s, W,
                    K, N, (int)fp4_blocks(K), out);
}

}  // namespace

cudaError_t launch_fp4_quantize(bool f32, const void* X, long long rows, int cols, long long ldx, const Fp4View& out,
                                cudaStream_t s) {
    RM_HOST_BOUNDS(X && rows >= 1 && cols >= 1 && ldx >= cols && fp4_holds(out, cols));
    return f32 ? quantize(static_cast<const float*>(X), rows, cols, ldx, out, s)
               : quantize(static_cast<const __nv_bfloat16*>(X), rows, cols, ldx, out, s);
}

cudaError_t launch_fp4_dequantize(const Fp4View& in, long long rows, int cols, void* Y, bool f32, long long ldy,
                                  cudaStream_t s) {
    RM_HOST_BOUNDS(Y && rows >= 1 && cols >= 1 && ldy >= cols && fp4_holds(in, cols));
    return f32 ? dequantize(in, rows, cols, static_cast<float*>(Y), ldy, s)
               : dequantize(in, rows, cols, static_cast<__nv_bfloat16*>(Y), ldy, s);
}

cudaError_t launch_fp4_quantize_weight(bool f32, const void* W, int G, int K, int N, const Fp4View& out, cudaStream_t s) {
    RM_HOST_BOUNDS(W && G >= 1 && G <= 65535 && K >= 1 && N >= 1 && out.lds == fp4_weight_quads(K) &&
                   fp8_on(out.codes, 16) && fp8_on(out.scales, 16) && out.ld % 16 == 0 && out.ld >= 16 * fp4_blocks(K));
    return f32 ? quantize_weight(static_cast<const float*>(W), G, K, N, out, s)
               : quantize_weight(static_cast<const __nv_bfloat16*>(W), G, K, N, out, s);
}

}  // namespace rm
