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
//   warps 4-11   epilogue: each thread owns one row's 128 columns, which is one
//                block of an 8-bit output: its largest value needs no exchange
// Tensor memory (512 columns): two accumulators of 256 columns that share 64,
// at columns 0 and 192, so that the next tile's product begins as soon as those
// 64 columns have been read, and a ring of four scale slots from column 448 (4
// columns for x's 128 rows, 8 for W's 256 columns).
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error
// word and all roles unwind.
#include <cudaTypedefs.h>

#include <mutex>

#include "rm_fp8.cuh"
#include "rm_fp8_tc.cuh"
#include "rm_train_math.cuh"

namespace rm {
namespace f8 {

constexpr int BM = 128;                  // rows (samples) per CTA
constexpr int BN = 256;                  // columns per tile
constexpr int BK = 128;                  // one scale block
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BN / 2 * BK;     // this CTA's half of the columns
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 5;
constexpr int SF_SLOTS = 4;
constexpr int SF_BYTES = 512 * 3;        // x: 128 rows, W: 2 x 128 columns
constexpr int EPI_WARPS = 8;
constexpr int STAGING = 4096;            // per epilogue warp: 32 rows of 128 bytes
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr uint32_t ACC1_COL = 192;       // the second accumulator's first column
constexpr int SF_COL = 448;
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_WARPS * STAGING + SF_SLOTS * SF_BYTES + 256;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
// registers: 384 threads launched with 168; 128 x 80 + 256 x 208 <= 384 x 168
constexpr int REGS_OTHER = 80, REGS_EPI = 208;

enum Epi { EPI_BF16, EPI_F32, EPI_GELU, EPI_GELU_KEEP, EPI_DGELU };

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
    void* y;                             // stored directly where the rows do not suit TMA
    bool direct;
    uint8_t* s0;                         // exponent bytes of the 8-bit outputs (GELU: a; DGELU: dU)
    uint8_t* s1;                         // GELU_KEEP: u
    long long s0_ld, s1_ld;
    const uint8_t* u;                    // DGELU: kept u's codes and exponent bytes
    const uint8_t* us;
    long long u_ld, us_ld;
    float* colpart;                      // DGELU: sums of dU over 32 rows, [T][m_tiles * 8][N]
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

// One row's 128 bytes into this warp's staging (128-byte swizzle: 16-byte piece
// c of row r at c ^ (r % 8)), four codes or two bf16 per word.
__device__ __forceinline__ void stage16(uint32_t stage, int lane, int c, uint32_t w0, uint32_t w1, uint32_t w2,
                                        uint32_t w3) {
    st_shared_v4(stage + 128u * lane + 16u * (uint32_t)(c ^ (lane & 7)), w0, w1, w2, w3);
}

// The staged 32 rows to their place: columns from n, samples from m.
__device__ __forceinline__ void store_staged(const CUtensorMap* map, uint32_t stage, int n, int m, int t, int lane,
                                             bool inside) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (inside) tma_store_3d(map, stage, n, m, t);
        bulk_commit_group();
    }
}
__device__ __forceinline__ void staging_free(int lane) {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
}

__device__ __forceinline__ float row_amax(const float (&v)[128]) {
    float m[4] = {};
#pragma unroll
    for (int i = 0; i < 128; ++i) m[i & 3] = fmaxf(m[i & 3], fabsf(v[i]));    // passes over NaN
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The row's 128 values in 8 bits: codes staged and stored, the exponent byte to *scale.
__device__ __forceinline__ void save_row(float (&v)[128], const CUtensorMap* map, uint32_t stage, uint8_t* scale,
                                         int n, int m_warp, int t, int lane, bool store, bool row_ok) {
    float amax = row_amax(v);
    if (amax == __int_as_float(0x7f800000)) {          // infinities become NaN and do not count
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = fp8_poison(v[i]);
        amax = row_amax(v);
    }
    const uint32_t E = fp8_exponent<false>(__float_as_uint(amax));
    const uint64_t s = f2_splat(fp8_inv_scale(E));
    staging_free(lane);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = 16 * c + 4 * j;
            float q[4];
            f2_unpack(f2_mul(f2_pack(v[i], v[i + 1]), s), q[0], q[1]);
            f2_unpack(f2_mul(f2_pack(v[i + 2], v[i + 3]), s), q[2], q[3]);
            w[j] = fp8_pack4<false>(q[0], q[1], q[2], q[3]);
        }
        stage16(stage, lane, c, w[0], w[1], w[2], w[3]);
    }
    store_staged(map, stage, n, m_warp, t, lane, store);
    if (row_ok) *scale = (uint8_t)E;
}

// Sum of v over the 32 lanes for each of 32 columns, column c in lane c.
__device__ __forceinline__ float column_sums(const float* v, int lane) {
    float w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = v[i];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = upper ? w[i] : w[i + o], keep = upper ? w[i + o] : w[i];
            w[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return w[0];
}

template <int EPI>
__device__ __forceinline__ void epilogue(float (&v)[128], const Args& a, const CUtensorMap* m0, const CUtensorMap* m1,
                                         const uint4 (&u8)[8], uint32_t u_byte, const Tile& tl, int m_warp, int n,
                                         int lane, uint32_t stage) {
    const int m = m_warp + lane;
    const bool row_ok = m < a.B && n < a.N, store = m_warp < a.B && n < a.N;
    const size_t row = (size_t)m * a.T + tl.t;
    if (EPI != EPI_DGELU && a.bias) {
        const float* b = a.bias + (size_t)tl.t * a.N + n;
        if (n + 128 <= a.N && (a.N & 3) == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float4 q = __ldg(reinterpret_cast<const float4*>(b) + i);
                v[4 * i] += q.x, v[4 * i + 1] += q.y, v[4 * i + 2] += q.z, v[4 * i + 3] += q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 128; ++i)
                if (n + i < a.N) v[i] += __ldg(b + i);
        }
    }
    if constexpr (EPI == EPI_BF16) {
        if (a.direct) {
            __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(a.y) + row * (size_t)a.N + n;
#pragma unroll
            for (int i = 0; i < 128; ++i)
                if (row_ok && n + i < a.N) y[i] = __float2bfloat16_rn(v[i]);
            return;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            staging_free(lane);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float* p = v + 64 * h + 8 * c;
                stage16(stage, lane, c, pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                        pack_bf16x2(p[6], p[7]));
            }
            store_staged(m0, stage, n + 64 * h, m_warp, tl.t, lane, store && n + 64 * h < a.N);
        }
    } else if constexpr (EPI == EPI_F32) {
        if (a.direct) {
            float* y = reinterpret_cast<float*>(a.y) + row * (size_t)a.N + n;
#pragma unroll
            for (int i = 0; i < 128; ++i)
                if (row_ok && n + i < a.N) y[i] = v[i];
            return;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            staging_free(lane);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float* p = v + 32 * h + 4 * c;
                stage16(stage, lane, c, __float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]),
                        __float_as_uint(p[3]));
            }
            store_staged(m0, stage, n + 32 * h, m_warp, tl.t, lane, store && n + 32 * h < a.N);
        }
    } else if constexpr (EPI == EPI_GELU || EPI == EPI_GELU_KEEP) {
        const int blk = n / kFp8Block;
        if constexpr (EPI == EPI_GELU_KEEP)
            save_row(v, m1, stage, a.s1 + row * (size_t)a.s1_ld + blk, n, m_warp, tl.t, lane, store, row_ok);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const uint64_t g = gelu_erf_x2(f2_pack(v[2 * i], v[2 * i + 1]), 0ull);
            f2_unpack(g, v[2 * i], v[2 * i + 1]);
        }
        save_row(v, m0, stage, a.s0 + row * (size_t)a.s0_ld + blk, n, m_warp, tl.t, lane, store, row_ok);
    } else {
        const float s = fp8_scale(u_byte);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t w[4] = {u8[c].x, u8[c].y, u8[c].z, u8[c].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = fp8_unpack2<false>(w[j >> 1] >> (16 * (j & 1)));
                uint64_t val, grad;
                gelu_with_grad_x2(f2_pack(f.x, f.y), f2_splat(s), 0ull, val, grad);
                float g0, g1;
                f2_unpack(grad, g0, g1);
                v[16 * c + 2 * j] *= g0;
                v[16 * c + 2 * j + 1] *= g1;
            }
        }
        // sums over this warp's 32 rows, for the bias gradient
        float* part = a.colpart + ((size_t)tl.t * a.m_tiles * 8 + m_warp / 32) * a.N;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float cs = column_sums(v + 32 * h, lane);
            if (n + 32 * h + lane < a.N) part[n + 32 * h + lane] = cs;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            staging_free(lane);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float* p = v + 64 * h + 8 * c;
                stage16(stage, lane, c, pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                        pack_bf16x2(p[6], p[7]));
            }
            store_staged(m1, stage, n + 64 * h, m_warp, tl.t, lane, store && n + 64 * h < a.N);
        }
        save_row(v, m0, stage, a.s0 + row * (size_t)a.s0_ld + n / kFp8Block, n, m_warp, tl.t, lane, store, row_ok);
    }
}

template <int EPI, bool TRANS>
__global__ void __launch_bounds__(THREADS, 1)
fp8_product_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1, const Args args) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    const uint32_t sA = base, sB = base + STAGES * A_BYTES;
    const uint32_t sEpi = base + STAGES * STAGE_BYTES;
    const uint32_t sSF = sEpi + EPI_WARPS * STAGING;
    const uint32_t bar0 = sSF + SF_SLOTS * SF_BYTES;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + SF_SLOTS + s); };
    auto tfull_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + x); };
    auto tempty_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + 2 + x); };
    const uint32_t shared_bar = bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + 4);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (shared_bar + 8u - base));
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
        mbar_init(shared_bar, EPI_WARPS);        // the even CTA's: the warps that own the shared columns
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc_pair(smem_u32(tmem_holder), 512);
        tmem_relinquish_pair();
    }
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
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t stage = sEpi + (uint32_t)(warp - 4) * STAGING;
        const uint32_t shared_leader = mapa_shared(shared_bar, 0);
        uint32_t phase = 0;
        int acc = 0;
        for (long long i = unit; i < args.tiles; i += nunits) {
            const Tile tl = tile_of(i, args);
            const int m_warp = tl.m0 + BM * (int)rank + 32 * quad, n = tl.n0 + 128 * half;
            uint4 u8[8];
            uint32_t u_byte = 127;
            if constexpr (EPI == EPI_DGELU) {        // the kept u, loaded while the product runs
                const bool here = m_warp + lane < args.B && n < args.N;
                const size_t row = (size_t)(m_warp + lane) * args.T + tl.t;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    u8[c] = here && n + 16 * c < args.N
                                ? __ldg(reinterpret_cast<const uint4*>(args.u + row * (size_t)args.u_ld + n) + c)
                                : make_uint4(0, 0, 0, 0);
                if (here) u_byte = __ldg(args.us + row * (size_t)args.us_ld + n / kFp8Block);
            }
            if (!wait_bounded(tfull_bar(acc), phase, abort_flag, args.err, args.timeout_ns)) break;
            tc_fence_after();
            // The whole row comes out at once, so the accumulator is free again long
            // before the epilogue is done; first of all the 64 columns that the other
            // accumulator shares (the last of accumulator 0, the first of 1).
            uint32_t r[4][32];
            const uint32_t tcol =
                tmem_base + ((uint32_t)(32 * quad) << 16) + (acc ? ACC1_COL : 0u) + 128u * half;
            auto load_half = [&](int h) {
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_ld32_nowait(tcol + 64u * h + 32u * c, r[2 * h + c]);
            };
            auto shared_out = [&]() {
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(shared_leader);
            };
            if (half == 1) {
                load_half(1);
                if (acc == 0) shared_out();
                load_half(0);
            } else {
                load_half(0);
                if (acc == 1) shared_out();
                load_half(1);
            }
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_bar(acc), 0));
            acc ^= 1;
            if (acc == 0) phase ^= 1u;
            float v[128];
#pragma unroll
            for (int c = 0; c < 128; ++c) v[c] = __uint_as_float(r[c >> 5][c & 31]);
            epilogue<EPI>(v, args, &tm0, &tm1, u8, u_byte, tl, m_warp, n, lane, stage);
        }
        if (lane == 0) bulk_wait_group<0>();         // this warp's tensor stores have landed
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
                    long long groups, long long row_bytes, long long group_bytes, int box_inner, int box_rows) {
    if (!f8::get_encoder()) return false;
    cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)groups};
    cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)group_bytes};
    cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return f8::g_encode(m, type, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace f8 {

template <int EPI, bool TRANS>
cudaError_t run(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& m0, const CUtensorMap& m1,
                const Args& a, int num_sms, cudaStream_t s) {
    auto k = fp8_product_kernel<EPI, TRANS>;
    cudaError_t e = smem_attr_once((const void*)k, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const long long pairs = num_sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (a.tiles < pairs ? a.tiles : pairs)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
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
    e = cudaLaunchKernelEx(&cfg, k, mx, mw, m0, m1, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int EPI>
cudaError_t run_either(bool trans, const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& m0,
                       const CUtensorMap& m1, const Args& a, int num_sms, cudaStream_t s) {
    return trans ? run<EPI, true>(mx, mw, m0, m1, a, num_sms, s) : run<EPI, false>(mx, mw, m0, m1, a, num_sms, s);
}

}  // namespace f8

int fp8_colpart_rows(int B) { return (B + 2 * f8::BM - 1) / (2 * f8::BM) * 8; }

cudaError_t launch_fp8_product(const Fp8Product& p, const Fp8Device& dev, cudaStream_t s) {
    using namespace f8;
    if (fp8_streams(p)) return launch_fp8_stream(p, dev, s);
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
    CUtensorMap mx, mw, m0, m1;
    const auto u8t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!fp8_tensor_map(&mx, u8t, p.x.codes, p.K, p.B, p.T, p.T * p.x.ld, p.x.ld, BK, BM) ||
        !fp8_tensor_map(&mw, u8t, p.w.codes, wc, wr, p.T, p.w.ld, (long long)wr * p.w.ld, 128, 128))
        return cudaErrorInvalidValue;
    m0 = m1 = mx;
    auto map8 = [&](CUtensorMap* m, const Fp8View& q) {
        return fp8_tensor_map(m, u8t, q.codes, p.N, p.B, p.T, p.T * q.ld, q.ld, 128, 32);
    };
    auto map16 = [&](CUtensorMap* m, void* q) {
        return fp8_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, p.N, p.B, p.T, 2ll * p.T * p.N, 2ll * p.N, 64, 32);
    };
    switch (p.epi) {
        case FP8_OUT_BF16:
            a.direct = p.N % 8 != 0;
            if (!a.direct && !map16(&m0, p.y)) return cudaErrorInvalidValue;
            return run_either<EPI_BF16>(p.trans, mx, mw, m0, m1, a, dev.num_sms, s);
        case FP8_OUT_F32:
            a.direct = p.N % 4 != 0;
            if (!a.direct && !fp8_tensor_map(&m0, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.y, p.N, p.B, p.T,
                                             4ll * p.T * p.N, 4ll * p.N, 32, 32))
                return cudaErrorInvalidValue;
            return run_either<EPI_F32>(p.trans, mx, mw, m0, m1, a, dev.num_sms, s);
        case FP8_GELU:
            if (p.trans || !map8(&m0, p.o0)) return cudaErrorInvalidValue;
            a.s0 = p.o0.scales, a.s0_ld = p.o0.lds;
            if (!p.o1.codes) return run<EPI_GELU, false>(mx, mw, m0, m1, a, dev.num_sms, s);
            if (!map8(&m1, p.o1)) return cudaErrorInvalidValue;
            a.s1 = p.o1.scales, a.s1_ld = p.o1.lds;
            return run<EPI_GELU_KEEP, false>(mx, mw, m0, m1, a, dev.num_sms, s);
        case FP8_DGELU:
            if (!p.trans || !map8(&m0, p.o0) || !map16(&m1, p.y)) return cudaErrorInvalidValue;
            a.s0 = p.o0.scales, a.s0_ld = p.o0.lds;
            a.u = p.o1.codes, a.u_ld = p.o1.ld, a.us = p.o1.scales, a.us_ld = p.o1.lds;
            a.colpart = p.colpart;
            return run<EPI_DGELU, true>(mx, mw, m0, m1, a, dev.num_sms, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace rm
