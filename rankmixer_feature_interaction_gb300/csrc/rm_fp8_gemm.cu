// Per-token products of 8-bit operands on the 5th-generation tensor cores:
//   Y[b][t][n] = sum_k x[b][t][k] W[t][k][n]   (or W[t][n][k])
// with one power-of-two scale per 128 values of x's rows and per 128 x 128
// values of W.  Power-of-two scales are what the block-scaled MMA
// (tcgen05.mma kind::mxf8f6f4) takes: it multiplies each 32-deep step's exact
// products by both operands' scales on the way into the float32 accumulator,
// so the sum over all of K stays in tensor memory and the CUDA cores are free
// for the epilogue (bias, GELU, its derivative, rounding to 8 bits).
//
// Kernel: one persistent pair of CTAs (two SMs) per 256 x 256 tile of one
// token, rows = samples; each CTA holds 128 rows of x and 128 columns of W per
// 128-deep k-block (32 KB a stage).
//   warp 0       TMA producer.  x: K-major (boxes of 128 bytes of K x 128
//                samples).  W [K][N]: MN-major (128 bytes of N x 128 of K);
//                W [N][K]: K-major.  One copy of W serves both directions.
//   warp 1       MMA issuer (the even CTA's)
//   warp 2       scales: a 32-bit word holds one row's exponent bytes of four
//                k-blocks, just as they lie in memory, so scales move once per
//                four k-blocks: lane l takes rows l, l + 32, l + 64, l + 96,
//                writes 16 bytes to shared memory, and the MMA issuer copies
//                512 bytes per 128 rows to tensor memory (tcgen05.cp)
//   warps 4-19   epilogue: each thread owns 64 columns of one row; a block of an
//                8-bit output is two threads', whose largest values meet in
//                shared memory.  Four warps per scheduler: with two (128 columns
//                a thread, no exchange) GELU and its rounding ran at 0.39
//                instructions per cycle, waiting for themselves
// Tensor memory (512 columns): two accumulators of 256 columns that share 64,
// at columns 0 and 192, so that the next tile's product begins as soon as those
// 64 columns have been read, and a ring of four scale slots from column 448 (4
// columns for x's 128 rows, 8 for W's 256 columns).
// Measured, T = 32, bf16 out: 4096 samples, 6144 to 1536 717 us (3.45 PFLOP/s), 1536
// to 6144 836 us (2.96, 12 k-blocks a tile); 1024 samples 205 and 230 us (on other
// GPUs up to 736 and 957 us at 4096).  Bound by the tensor cores, which the power limit
// slows at the large sizes, and where a tile has few k-blocks by what lies between two
// tiles (the shared columns); with an 8-bit
// output and Gelu or its derivative, by the epilogue's instructions beside them (50
// and 45% of the tensor pipe's cycles against 68).
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error
// word and all roles unwind.
#include <cudaTypedefs.h>

#include <mutex>

#include "rm_fp8.cuh"
#include "rm_fp8_tc.cuh"

namespace rm {
namespace f8 {

constexpr int BM = 128;                  // rows (samples) per CTA
constexpr int BN = 256;                  // columns per tile
constexpr int BK = 128;                  // one scale block
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BN / 2 * BK;     // this CTA's half of the columns
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int SF_SLOTS = 4;
constexpr int SF_BYTES = 512 * 3;        // x: 128 rows, W: 2 x 128 columns
constexpr int EPI_WARPS = 16;
constexpr int COLS = 64;                 // columns per epilogue warp
constexpr int STAGING = 2048;            // per epilogue warp: 32 rows of 64 bytes
constexpr int RED_BYTES = 2 * 2 * EPI_WARPS * 32 * 4;   // rows' largest values: [tile parity][output][warp][row]
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr uint32_t ACC1_COL = 192;       // the second accumulator's first column
constexpr int SF_COL = 448;
// registers: 640 threads launched with 96; 128 x 56 + 512 x 104 <= 640 x 96
constexpr int REGS_OTHER = 56, REGS_EPI = 104;

enum Epi { EPI_BF16, EPI_F32, EPI_GELU, EPI_GELU_KEEP, EPI_DGELU };

// Shared memory: the stages, 2 KB of staging per epilogue warp, the scale slots;
// for DGELU 2 KB more per epilogue warp for the next tile's kept u and the table of
// Gelu', and a stage less.
constexpr int TAB_LO = 127 - 33, TAB_ROWS = 38, TAB_BYTES = TAB_ROWS * 128 * 4;
template <int EPI>
struct Cfg {
    static constexpr int STAGES = EPI == EPI_DGELU ? 4 : 5;
    static constexpr int U_BYTES = EPI == EPI_DGELU ? EPI_WARPS * STAGING : 0;
    static constexpr int TAB = EPI == EPI_DGELU ? TAB_BYTES : 0;
    static constexpr int SMEM_BYTES =
        1024 + STAGES * STAGE_BYTES + EPI_WARPS * STAGING + U_BYTES + SF_SLOTS * SF_BYTES + RED_BYTES + TAB + 512;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
};

struct Args {
    int B, T, K, N;
    int m_tiles, n_tiles, kblocks;
    long long tiles;
    const uint8_t* xs;                   // x's exponent bytes: row (b, t) at (b T + t) xs_ld
    long long xs_ld;
    const uint8_t* ws;                   // W's: block row r of token t at (t w_rows + r) ws_ld
    long long ws_ld;
    int w_rows;
    uint32_t x_format;                   // 0 e4m3, 1 e5m2
    const float* bias;                   // [T][N] or null
    void* y;                             // [B][T][N]
    bool vec;                            // y's rows are 16-byte aligned
    Fp8View o0, o1;                      // GELU: a, u (kept); DGELU: dU, the kept u
    int* err;
    unsigned long long timeout_ns;
};

struct Tile {
    int t, m0, n0;
};
// M tiles fastest: neighbouring pairs share W's columns, and a token's x (which
// every column tile reads again) stays in L2.
__device__ __forceinline__ Tile tile_of(long long i, const Args& a) {
    const int per = a.m_tiles * a.n_tiles;
    Tile r;
    r.t = (int)(i / per);
    const int rem = (int)(i - (long long)r.t * per), nb = rem / a.m_tiles;
    r.m0 = (rem - nb * a.m_tiles) * 2 * BM;
    r.n0 = nb * BN;
    return r;
}

// Where the two warps of a block meet: this warp's and the partner's rows of the
// exchange (written once per tile and output, and read before the partner can
// write them again two tiles later) and a barrier of two arrivals, bounded as all.
struct Partner {
    volatile float* mine;
    const volatile float* theirs;
    uint32_t bar, phase;
    volatile int* abort;
};

// Largest magnitude of the row's block, this thread's half and its partner's;
// passes over NaN.  False when the wait ran out.
__device__ __forceinline__ float half_amax(const float (&v)[COLS]) {
    float m[2] = {};
#pragma unroll
    for (int i = 0; i < COLS; i += 2) m[i >> 1 & 1] = max3(m[i >> 1 & 1], fabsf(v[i]), fabsf(v[i + 1]));
    return fmaxf(m[0], m[1]);
}
__device__ __forceinline__ bool block_amax(float (&v)[COLS], Partner& p, int which, const Args& a, int lane, float& amax) {
    float m = half_amax(v);
    if (m == __int_as_float(0x7f800000)) {             // infinities become NaN and do not count
#pragma unroll
        for (int i = 0; i < COLS; ++i) v[i] = fp8_poison(v[i]);
        m = half_amax(v);
    }
    p.mine[which * EPI_WARPS * 32 + lane] = m;
    __syncwarp();
    if (lane == 0) mbar_arrive(p.bar);
    if (!wait_bounded(p.bar, p.phase, p.abort, a.err, a.timeout_ns)) return false;
    p.phase ^= 1u;
    amax = fmaxf(m, p.theirs[which * EPI_WARPS * 32 + lane]);
    return true;
}

// The row's 64 values in 8 bits to columns n on of `out`; the warp with a block's
// first half also writes its exponent bytes.
__device__ __forceinline__ void save_row(const float (&v)[COLS], float amax, const Fp8View& out, const Args& a, int t,
                                         int m_warp, int n, int rows, int lane, uint32_t stage) {
    const uint32_t E = fp8_exponent<false>(__float_as_uint(amax));
    const uint64_t s = f2_splat(fp8_inv_scale(E));
#pragma unroll
    for (int c = 0; c < COLS / 16; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = 16 * c + 4 * j;
            float q[4];
            f2_unpack(f2_mul(f2_pack(v[i], v[i + 1]), s), q[0], q[1]);
            f2_unpack(f2_mul(f2_pack(v[i + 2], v[i + 3]), s), q[2], q[3]);
            w[j] = fp8_pack4<false>(q[0], q[1], q[2], q[3]);
        }
        st_shared_v4(staged_at(stage, lane, c), w[0], w[1], w[2], w[3]);
    }
    const size_t row = (size_t)m_warp * a.T + t;
    store_rows<true, 1>(stage, reinterpret_cast<char*>(out.codes) + row * (size_t)out.ld + n,
                        (size_t)a.T * (size_t)out.ld, rows, a.N - n, lane);
    if (n % kFp8Block == 0 && lane < rows)
        out.scales[(row + (size_t)lane * a.T) * (size_t)out.lds + n / kFp8Block] = (uint8_t)E;
}

// 64 bytes of each row of Y from column n on.
template <typename OUT>
__device__ __forceinline__ void save_piece(const float* v, const Args& a, int t, int m_warp, int n, int rows, int lane,
                                           uint32_t stage) {
    constexpr int E = sizeof(OUT);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if constexpr (E == 2)
            st_shared_v4(staged_at(stage, lane, c), pack_bf16x2(v[8 * c], v[8 * c + 1]),
                         pack_bf16x2(v[8 * c + 2], v[8 * c + 3]), pack_bf16x2(v[8 * c + 4], v[8 * c + 5]),
                         pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
        else
            st_shared_v4(staged_at(stage, lane, c), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                         __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
    }
    char* dst = reinterpret_cast<char*>(a.y) + (((size_t)m_warp * a.T + t) * (size_t)a.N + n) * E;
    const size_t pitch = (size_t)a.T * (size_t)a.N * E;
    const int bytes = min(a.N - n, 64) * E;            // the row's rest may be more bytes than fit 32 bits
    if (a.vec)
        store_rows<true, E>(stage, dst, pitch, rows, bytes, lane);
    else
        store_rows<false, E>(stage, dst, pitch, rows, bytes, lane);
}

template <int EPI>
__device__ __forceinline__ bool epilogue(float (&v)[COLS], const Args& a, const Tile& tl, int m_warp, int n, int lane,
                                         uint32_t stage, Partner& partner) {
    const int rows = n < a.N ? min(32, a.B - m_warp) : 0;        // this warp's rows that exist (may be negative)
    if (EPI != EPI_DGELU && a.bias) {                  // brought to the staging before the tile was waited for
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) {
            float4 q;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w)
                         : "r"(stage + 16u * i));
            f2_unpack(f2_add(f2_pack(v[4 * i], v[4 * i + 1]), f2_pack(q.x, q.y)), v[4 * i], v[4 * i + 1]);
            f2_unpack(f2_add(f2_pack(v[4 * i + 2], v[4 * i + 3]), f2_pack(q.z, q.w)), v[4 * i + 2], v[4 * i + 3]);
        }
        __syncwarp();
    }
    if constexpr (EPI == EPI_BF16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            save_piece<__nv_bfloat16>(v + 32 * h, a, tl.t, m_warp, n + 32 * h, rows, lane, stage);
    } else if constexpr (EPI == EPI_F32) {
#pragma unroll
        for (int h = 0; h < 4; ++h) save_piece<float>(v + 16 * h, a, tl.t, m_warp, n + 16 * h, rows, lane, stage);
    } else if constexpr (EPI == EPI_GELU || EPI == EPI_GELU_KEEP) {
        if constexpr (EPI == EPI_GELU_KEEP) {
            float m;
            if (!block_amax(v, partner, 1, a, lane, m)) return false;
            save_row(v, m, a.o1, a, tl.t, m_warp, n, rows, lane, stage);
        }
#pragma unroll
        for (int i = 0; i < COLS; ++i) v[i] = fp8_gelu(v[i]);
        float m;
        if (!block_amax(v, partner, 0, a, lane, m)) return false;
        save_row(v, m, a.o0, a, tl.t, m_warp, n, rows, lane, stage);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            save_piece<__nv_bfloat16>(v + 32 * h, a, tl.t, m_warp, n + 32 * h, rows, lane, stage);
        float m;
        if (!block_amax(v, partner, 0, a, lane, m)) return false;
        save_row(v, m, a.o0, a, tl.t, m_warp, n, rows, lane, stage);
    }
    return true;
}

// Gelu'(u) of a kept u depends on 8 bits and an exponent, so a table in shared
// memory holds it: Gelu'(u) - 1/2, an odd function, for the 128 magnitudes under
// every exponent byte from TAB_LO on, built once by each CTA.  Below TAB_LO |u| is
// so small that the lowest row is right to 4e-8; blocks above the last row (|u|
// up to 7168) are computed.  Seven instructions a value where the formula takes 18.
__device__ __forceinline__ void build_table(float* tab, int i, int n) {
    for (; i < TAB_ROWS * 128; i += n)
        tab[i] = fp8_gelu_grad(fp8_unpack2<false>((uint32_t)i & 127u).x * fp8_scale(TAB_LO + (i >> 7))) - 0.5f;
}

// v *= Gelu'(u), u the row's 64 codes in shared memory under exponent byte E.
__device__ __forceinline__ void times_gelu_grad(float (&v)[COLS], uint32_t codes, uint32_t E, uint32_t tab, int lane) {
    if (E < TAB_LO + TAB_ROWS) {
        const uint32_t row = tab + 512u * (max(E, (uint32_t)TAB_LO) - TAB_LO);
#pragma unroll
        for (int c = 0; c < COLS / 16; ++c) {
            const uint4 q = staged16(codes, lane, c);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t x = w[j >> 2];
                const int k = 8 * (j & 3);
                uint32_t h;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(h) : "r"(row + ((k ? x >> (k - 2) : x << 2) & 0x1fcu)));
                const float g = __uint_as_float(h ^ (x << (24 - k) & 0x80000000u));
                v[16 * c + j] = fmaf(v[16 * c + j], g, 0.5f * v[16 * c + j]);
            }
        }
    } else {
        const float scale = fp8_scale(E);
#pragma unroll
        for (int c = 0; c < COLS / 16; ++c) {
            const uint4 q = staged16(codes, lane, c);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = fp8_unpack2<false>(w[j >> 1] >> (16 * (j & 1)));
                v[16 * c + 2 * j] *= fp8_gelu_grad(f.x * scale);
                v[16 * c + 2 * j + 1] *= fp8_gelu_grad(f.y * scale);
            }
        }
    }
}

template <int EPI, bool TRANS>
__global__ void __launch_bounds__(THREADS, 1)
fp8_product_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmU, const Args args) {
    constexpr int STAGES = Cfg<EPI>::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    const uint32_t sA = base, sB = base + STAGES * A_BYTES;
    const uint32_t sEpi = base + STAGES * STAGE_BYTES;
    const uint32_t sU = sEpi + EPI_WARPS * STAGING, sSF = sU + Cfg<EPI>::U_BYTES;
    float* red = reinterpret_cast<float*>(base_ptr + (sSF - base) + SF_SLOTS * SF_BYTES);
    float* tab = red + RED_BYTES / 4;
    const uint32_t bar0 = sSF + SF_SLOTS * SF_BYTES + RED_BYTES + Cfg<EPI>::TAB;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + SF_SLOTS + s); };
    auto tfull_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + x); };
    auto tempty_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + 2 + x); };
    const uint32_t shared_bar = bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + 4);
    auto u_bar = [&](int w) { return shared_bar + 8u + 8u * w; };
    auto pair_bar = [&](int w) { return shared_bar + 8u + 8u * (EPI_WARPS + w); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (pair_bar(EPI_WARPS / 2) - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const long long unit = blockIdx.x >> 1, nunits = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);           // the even CTA's: its producer, expecting both CTAs' bytes
            mbar_init(empty_bar(s), 1);          // multicast commit
        }
        for (int s = 0; s < SF_SLOTS; ++s) {
            mbar_init(sfull_bar(s), 2);          // the even CTA's: both CTAs' scale warps
            mbar_init(sempty_bar(s), 1);         // multicast commit
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(tfull_bar(x), 1);              // multicast commit
            mbar_init(tempty_bar(x), 2 * EPI_WARPS); // the even CTA's: every epilogue warp of both CTAs
        }
        for (int w = 0; w < EPI_WARPS; ++w) mbar_init(u_bar(w), 1);
        for (int w = 0; w < EPI_WARPS / 2; ++w) mbar_init(pair_bar(w), 2);
        mbar_init(shared_bar, 2 * EPI_WARPS / 4);    // the even CTA's: the warps that own the shared columns
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
    if constexpr (EPI == EPI_DGELU)
        if (warp >= 4) build_table(tab, threadIdx.x - 128, 32 * EPI_WARPS);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
    const int kblocks = args.kblocks;
    pdl_wait();
    pdl_launch_next();

    if (warp < 4) {
        regs_dec<REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------ TMA producer ------------------------------
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (long long i = unit; ok && i < args.tiles; i += nunits) {
                const Tile tl = tile_of(i, args);
                const int xrow = tl.m0 + BM * (int)rank, wcol = tl.n0 + BN / 2 * (int)rank;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t fb = mapa_shared(full_bar(stage), 0);
                        if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2u * STAGE_BYTES);
                        tma_load_3d_pair(&tmX, sA + stage * A_BYTES, fb, kb * BK, xrow, tl.t);
                        if (TRANS)
                            tma_load_3d_pair(&tmW, sB + stage * B_BYTES, fb, kb * BK, wcol, tl.t);
                        else
                            tma_load_3d_pair(&tmW, sB + stage * B_BYTES, fb, wcol, kb * BK, tl.t);
                    }
                    __syncwarp();
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------ MMA issuer --------------------------------
            const uint32_t idesc = idesc_mxf8(2 * BM, BN, false, !TRANS) | (args.x_format << 7);
            constexpr uint32_t b_step = TRANS ? 32u : 32u * 128u;      // 32 values of K further
            const uint64_t a_desc = sw128_operand(sA, 16u), b_desc = sw128_operand(sB, TRANS ? 16u : (uint32_t)B_BYTES);
            int stage = 0, slot = 0;
            uint32_t phase = 0, sphase = 0, aphase = 0, cphase = 0;
            int acc = 0;
            bool ok = true;
            for (long long i = unit; ok && i < args.tiles; i += nunits) {
                // this accumulator's last tile is out, and of the other's tile the shared columns
                if (!wait_bounded(tempty_bar(acc), aphase ^ 1u, abort_flag, args.err, args.timeout_ns) ||
                    !wait_bounded(shared_bar, cphase ^ 1u, abort_flag, args.err, args.timeout_ns))
                    break;
                cphase ^= 1u;
                tc_fence_after();
                const uint32_t d = tmem_base + (acc ? ACC1_COL : 0u);
                for (int kb = 0; kb < kblocks; ++kb) {
                    const uint32_t sf = tmem_base + SF_COL + 16u * slot;
                    if ((kb & 3) == 0) {
                        if (!wait_bounded(sfull_bar(slot), sphase, abort_flag, args.err, args.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t src = sSF + slot * SF_BYTES;
                            copy_scales<true>(sf, scale_desc(src));
                            copy_scales<true>(sf + 4, scale_desc(src + 512));
                            copy_scales<true>(sf + 8, scale_desc(src + 1024));
                        }
                        __syncwarp();
                    }
                    if (!wait_bounded(full_bar(stage), phase, abort_flag, args.err, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const bool last = (kb & 3) == 3 || kb + 1 == kblocks;
                    if (elect_one()) {
                        const uint32_t id = with_scale_id(idesc, (uint32_t)(kb & 3));
                        const uint64_t a = a_desc + (uint32_t)(stage * (A_BYTES >> 4));
                        const uint64_t b = b_desc + (uint32_t)(stage * (B_BYTES >> 4));
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            umma_mxf8<true>(d, a + 2u * k, b + (b_step >> 4) * k, id, sf, sf + 4,
                                            (kb | k) != 0 ? 1u : 0u);
                        umma_commit_pair_mc(empty_bar(stage), (uint16_t)0x3);
                        if (last) umma_commit_pair_mc(sempty_bar(slot), (uint16_t)0x3);
                    }
                    __syncwarp();
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                    if (last && ++slot == SF_SLOTS) slot = 0, sphase ^= 1u;
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair_mc(tfull_bar(acc), (uint16_t)0x3);
                __syncwarp();
                acc ^= 1;
                if (acc == 0) aphase ^= 1u;
            }
        } else if (warp == 2) {
            // ------------------------------ scales ------------------------------------
            // one group of four k-blocks ahead: its words are loaded while the slot
            // of the current one is waited for
            const int groups = (kblocks + 3) / 4;
            struct Words {
                uint32_t x[4], w[2];
            };
            auto load = [&](const Tile& tl, int g) {
                Words r;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int m = tl.m0 + BM * (int)rank + 32 * j + lane;
                    r.x[j] = 0x7f7f7f7fu;
                    if (m < args.B)
                        r.x[j] = __ldg(reinterpret_cast<const uint32_t*>(
                                           args.xs + ((size_t)m * args.T + tl.t) * (size_t)args.xs_ld) + g);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int nb = tl.n0 / 128 + h;
                    r.w[h] = 0x7f7f7f7fu;
                    if (nb * 128 < args.N) {
                        if (TRANS) {
                            r.w[h] = __ldg(reinterpret_cast<const uint32_t*>(
                                               args.ws + ((size_t)tl.t * args.w_rows + nb) * (size_t)args.ws_ld) + g);
                        } else {
                            uint32_t v = 0;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int kb = 4 * g + q < kblocks ? 4 * g + q : kblocks - 1;
                                v |= (uint32_t)__ldg(args.ws + ((size_t)tl.t * args.w_rows + kb) * (size_t)args.ws_ld +
                                                     nb) << (8 * q);
                            }
                            r.w[h] = v;
                        }
                    }
                }
                return r;
            };
            int slot = 0, g = 0;
            uint32_t phase = 0;
            long long i = unit;
            Words now{};
            if (i < args.tiles) now = load(tile_of(i, args), 0);
            while (i < args.tiles) {
                if (++g == groups) g = 0, i += nunits;
                Words next{};
                if (i < args.tiles) next = load(tile_of(i, args), g);
                if (!wait_bounded(sempty_bar(slot), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) break;
                const uint32_t dst = sSF + slot * SF_BYTES + 16u * lane;
                st_shared_v4(dst, now.x[0], now.x[1], now.x[2], now.x[3]);
                st_shared_v4(dst + 512, now.w[0], now.w[0], now.w[0], now.w[0]);
                st_shared_v4(dst + 1024, now.w[1], now.w[1], now.w[1], now.w[1]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(mapa_shared(sfull_bar(slot), 0));
                if (++slot == SF_SLOTS) slot = 0, phase ^= 1u;
                now = next;
            }
        }
    } else {
        // ------------------------------ epilogue --------------------------------------
        regs_inc<REGS_EPI>();
        const int quad = warp & 3, part = (warp - 4) >> 2;       // 32 rows, 64 columns
        const uint32_t stage = sEpi + (uint32_t)(warp - 4) * STAGING;
        const uint32_t shared_leader = mapa_shared(shared_bar, 0);
        Partner partner{nullptr, nullptr, pair_bar(4 * (part >> 1) + quad), 0, abort_flag};
        uint32_t phase = 0, uphase = 0, u_next = 127;
        int acc = 0;
        // DGELU: a tile's kept u is on its way while the tile before is worked on
        const uint32_t u_codes = sU + (uint32_t)(warp - 4) * STAGING, ub = u_bar(warp - 4);
        auto fetch_u = [&](long long i) {
            const Tile tl = tile_of(i, args);
            const int m = tl.m0 + BM * (int)rank + 32 * quad, n = tl.n0 + COLS * part;
            if (lane == 0) {
                mbar_arrive_expect_tx(ub, STAGING);
                tma_load_3d(&tmU, u_codes, ub, n, m, tl.t);
            }
            u_next = 127;
            if (m + lane < args.B && n < args.N)
                u_next = __ldg(args.o1.scales + ((size_t)(m + lane) * args.T + tl.t) * (size_t)args.o1.lds + n / kFp8Block);
        };
        if constexpr (EPI == EPI_DGELU) {
            if (unit < args.tiles) fetch_u(unit);
        }
        for (long long i = unit; i < args.tiles; i += nunits) {
            const Tile tl = tile_of(i, args);
            const int m_warp = tl.m0 + BM * (int)rank + 32 * quad, n = tl.n0 + COLS * part;
            if (EPI != EPI_DGELU && args.bias) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = n + 32 * h + lane;
                    const float b = c < args.N ? __ldg(args.bias + (size_t)tl.t * args.N + c) : 0.f;
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + 128u * h + 4u * lane), "f"(b) : "memory");
                }
                __syncwarp();
            }
            if (!wait_bounded(tfull_bar(acc), phase, abort_flag, args.err, args.timeout_ns)) break;
            tc_fence_after();
            // A thread's columns come out at once, so the accumulator is free again long
            // before the epilogue is done; the 64 columns that the other accumulator
            // shares are the last of accumulator 0 and the first of 1.
            uint32_t r[2][32];
            const uint32_t tcol =
                tmem_base + ((uint32_t)(32 * quad) << 16) + (acc ? ACC1_COL : 0u) + (uint32_t)(COLS * part);
            tmem_ld32_nowait(tcol, r[0]);
            tmem_ld32_nowait(tcol + 32u, r[1]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (part == (acc ? 0 : 3)) mbar_arrive_pair(shared_leader);
                mbar_arrive_pair(mapa_shared(tempty_bar(acc), 0));
            }
            float v[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) v[c] = __uint_as_float(r[c >> 5][c & 31]);
            if constexpr (EPI == EPI_DGELU) {
                if (!wait_bounded(ub, uphase, abort_flag, args.err, args.timeout_ns)) break;
                uphase ^= 1u;
                times_gelu_grad(v, u_codes, u_next, smem_u32(tab), lane);
                __syncwarp();
                if (i + nunits < args.tiles) fetch_u(i + nunits);
            }
            partner.mine = red + (acc * 2 * EPI_WARPS + (warp - 4)) * 32;
            partner.theirs = partner.mine + ((part & 1) ? -128 : 128);
            if (!epilogue<EPI>(v, args, tl, m_warp, n, lane, stage, partner)) break;
            acc ^= 1;
            if (acc == 0) phase ^= 1u;
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();    // no CTA leaves while its peer may still touch its memory
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
std::mutex g_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

bool get_encoder() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_encode) return true;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return false;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return true;
}

}  // namespace f8

bool fp8_tensor_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, long long inner, long long rows,
                    long long groups, long long row_bytes, long long group_bytes, int box_inner, int box_rows,
                    bool plain) {
    if (!f8::get_encoder()) return false;
    cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)groups};
    cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)group_bytes};
    cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return f8::g_encode(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        plain ? CU_TENSOR_MAP_SWIZZLE_NONE
                        : box_inner == 64 && type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                                   : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace f8 {

template <int EPI, bool TRANS>
cudaError_t run(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& mu, const Args& a, int num_sms,
                cudaStream_t s) {
    auto k = fp8_product_kernel<EPI, TRANS>;
    constexpr int smem = Cfg<EPI>::SMEM_BYTES;
    cudaError_t e = smem_attr_once((const void*)k, smem);
    if (e != cudaSuccess) return e;
    const long long pairs = num_sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (a.tiles < pairs ? a.tiles : pairs)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, k, mx, mw, mu, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace f8

cudaError_t launch_fp8_product(const Fp8Product& p, const Fp8Device& dev, cudaStream_t s) {
    using namespace f8;
    RM_HOST_BOUNDS(p.B >= 1 && p.T >= 1 && p.K >= 1 && p.N >= 1 && fp8_holds(p.x, p.K) && !p.w.e5m2);
    RM_HOST_BOUNDS(fp8_holds(p.w, p.trans ? p.K : p.N) && (!p.bias || fp8_on(p.bias, 16)));
    RM_HOST_BOUNDS(p.epi == FP8_GELU || fp8_on(p.y, 16));
    RM_HOST_BOUNDS(p.epi == FP8_OUT_BF16 || p.epi == FP8_OUT_F32 || (p.N % 16 == 0 && fp8_holds(p.o0, p.N)));
    RM_HOST_BOUNDS(p.epi == FP8_DGELU || p.o1.codes ? fp8_holds(p.o1, p.N) && !p.o1.e5m2 : true);
    if (fp8_streams(p, dev)) return launch_fp8_stream(p, dev, s);
    Args a{};
    a.B = p.B, a.T = p.T, a.K = p.K, a.N = p.N;
    a.m_tiles = (p.B + 2 * BM - 1) / (2 * BM);
    a.n_tiles = (p.N + BN - 1) / BN;
    a.kblocks = (p.K + BK - 1) / BK;
    a.tiles = (long long)p.T * a.m_tiles * a.n_tiles;
    a.xs = p.x.scales, a.xs_ld = p.x.lds;
    a.ws = p.w.scales, a.ws_ld = p.w.lds;
    const int wr = p.trans ? p.N : p.K, wc = p.trans ? p.K : p.N;
    a.w_rows = (wr + kFp8Block - 1) / kFp8Block;
    a.x_format = p.x.e5m2 ? 1u : 0u;
    a.bias = p.bias;
    a.y = p.y;
    a.err = dev.err;
    a.timeout_ns = dev.timeout_ns;
    a.o0 = p.o0, a.o1 = p.o1;
    a.vec = p.N % (p.epi == FP8_OUT_F32 ? 4 : 8) == 0;
    CUtensorMap mx, mw;
    const auto u8t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!fp8_tensor_map(&mx, u8t, p.x.codes, p.K, p.B, p.T, p.T * p.x.ld, p.x.ld, BK, BM) ||
        !fp8_tensor_map(&mw, u8t, p.w.codes, wc, wr, p.T, p.w.ld, (long long)wr * p.w.ld, 128, 128))
        return cudaErrorInvalidValue;
    const int sms = dev.num_sms;
    switch (p.epi) {
        case FP8_OUT_BF16:
            return p.trans ? run<EPI_BF16, true>(mx, mw, mx, a, sms, s) : run<EPI_BF16, false>(mx, mw, mx, a, sms, s);
        case FP8_OUT_F32:
            return p.trans ? run<EPI_F32, true>(mx, mw, mx, a, sms, s) : run<EPI_F32, false>(mx, mw, mx, a, sms, s);
        case FP8_GELU:
            if (p.trans) return cudaErrorNotSupported;
            return p.o1.codes ? run<EPI_GELU_KEEP, false>(mx, mw, mx, a, sms, s)
                              : run<EPI_GELU, false>(mx, mw, mx, a, sms, s);
        case FP8_DGELU: {
            CUtensorMap mu;
            if (!p.trans || !fp8_tensor_map(&mu, u8t, p.o1.codes, p.N, p.B, p.T, p.T * p.o1.ld, p.o1.ld, COLS, 32))
                return cudaErrorInvalidValue;
            return run<EPI_DGELU, true>(mx, mw, mu, a, sms, s);
        }
    }
    return cudaErrorNotSupported;
}

}  // namespace rm
