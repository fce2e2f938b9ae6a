// Products of 4-bit operands on the 5th-generation tensor cores:
//   Y[row][n] = sum_k x[row][k] W[g][n][k]    for the rows of every group g,
// groups being the tokens of a sample-major batch, or the experts of sorted rows.
// One power-of-two scale per 32 values of K of either operand, which the
// block-scaled MMA (tcgen05.mma kind::mxf4, 64 values of K a step) multiplies in on
// the way into the float32 accumulator; both operands K-major, as that kind has it.
//
// Kernel: one persistent pair of CTAs (two SMs) per 256 x 256 tile of one group;
// each CTA holds 128 rows of x and 128 rows (columns of Y) of W per k-block of 256
// values, 32 KB of codes a stage and 3 KB of exponent bytes.
//   warp 0       TMA producer: codes of x and W, W's exponent bytes (already in the
//                tensor cores' order, those of all 256 columns in both CTAs)
//   warp 1       MMA issuer (the even CTA's): six copies of exponent bytes to tensor
//                memory and four MMAs a k-block
//   warps 2, 3   x's exponent bytes (RowScales), every other step of two k-blocks
//   warps 4-19   epilogue, two groups of eight warps for every other tile, so that one
//                group's waits and reads lie beside the other's arithmetic (all sixteen
//                on one tile: layer 1 at B = 2048 290 us instead of 270).  A warp owns 32
//                rows and 128 columns, a thread 32 of one row at a time, which is a block
//                of a 4-bit output
// Tensor memory (512 columns): two accumulators of 256 columns that share 64, at
// columns 0 and 192, so that the next tile's product begins as soon as those 64
// columns have been read (first), and two slots of exponent bytes from column 448 (8
// columns for x, 16 for W).  Copies and MMAs of one thread run in order, so the slots
// need no barriers of their own.
// Measured, T = 32, 4096 samples, bf16 out: 6144 to 1536 337 us (7.3 PFLOP/s), 1536 to
// 6144 446 us (5.5; float32 out 610, 3.2 GB written); T = 4, 12288 to 6144 311 us (7.9).
// With many k-blocks bound by the tensor core and by what the SMs take in from L2: 35 KB
// of a CTA in 512 cycles, 68 bytes a cycle (6144 to 1536 303 us without an epilogue, 282
// with half of the operands too).  With few by the outputs on their way to memory: 1536 to
// 6144 takes 353 us without their stores and 325 without an epilogue; loads wait behind
// them, so a stage less costs 10%, and buffers for two pieces of a warp's outputs in its
// place gain nothing.  With Gelu (2048 samples: 252 us, 195 without) by accumulators that stay
// taken for most of their epilogue: the issuer waits for one 3010 of a tile's 6430 cycles,
// while neither the issue slots (58%) nor the tensor pipe (44%) are full.
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error
// word and all roles unwind.
#include <cudaTypedefs.h>

#include "rm_fp4_tc.cuh"

namespace rm {
namespace f4 {

constexpr int BM = 128;                  // rows per CTA
constexpr int BN = 256;                  // columns per tile
constexpr int A_BYTES = BM * 128, B_BYTES = BN / 2 * 128, SFB_BYTES = 2 * SF_BYTES;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int TX_BYTES = STAGE_BYTES + SFB_BYTES;       // what TMA brings to a CTA's stage
constexpr int STAGES = 5;
constexpr int EPI_WARPS = 16, GROUP_WARPS = 8;
constexpr int WARP_COLS = 128, CHUNK = 32;      // columns of a warp, and of a thread at a time
constexpr int STAGING = 2048;            // per epilogue warp: 32 rows of 64 bytes
constexpr int BIAS_BYTES = 2 * CHUNK * 4;       // per epilogue warp
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr uint32_t BAND = 8;             // tiles
constexpr uint32_t ACC1_COL = 192;       // the second accumulator's first column
constexpr uint32_t SF_COL = 448, SF_COLS = 24;
// registers: 640 threads launched with 96; 128 x 64 + 512 x 104 = 640 x 96
constexpr int REGS_OTHER = 64, REGS_EPI = 104;
using Scales = RowScales<BM, 3>;        // of each of the two warps
constexpr int SMEM_BYTES = 1024 + STAGES * (STAGE_BYTES + SF_BYTES + SFB_BYTES) + EPI_WARPS * (STAGING + BIAS_BYTES) +
                           2 * Scales::BYTES + 256;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

struct Args {
    int B, G, N;                         // rows of a group (per token), groups
    int m_tiles, n_tiles, kblocks, nb;
    uint32_t units;                      // tiles (per token; experts: the table's length times n_tiles)
    const int4* table;                   // experts: the tiles of rows (null: per token)
    long long n;                         // experts: rows that exist
    long long step;                      // between rows of a group
    const uint8_t* xs;
    long long xs_ld;
    const float* bias;                   // [G][N] or null
    void* y;
    bool vec;                            // y's rows are 16-byte aligned
    bool tma;                            // and no longer than 2^31 bytes, TMA's coordinates
    Fp4View o;
    int* err;
    unsigned long long timeout_ns;
};

// Rows m0 .. of group g (per token: samples; experts: sorted rows), columns n0 ..
struct Tile {
    int g, m0, rows, n0;
};
// Per token by bands of columns, in a band columns fastest: W's columns and a token's x
// stay in L2, and a row's outputs are written next to each other.  Bands of 8 tiles: 1536
// to 6144, 4096 samples 446 us, of one 460, of all 448 (and 16,384 to 16,384 686 us, not
// 530).  Gelu's outputs are few, and its registers too: of one tile.  Experts: columns fastest,
// so that a tile of rows is read from memory once.
template <bool EXPERTS, bool GELU>
__device__ __forceinline__ Tile tile_of(uint32_t i, const Args& a) {
    Tile t;
    if (EXPERTS) {
        const uint32_t l = i / (uint32_t)a.n_tiles;
        t.n0 = (int)(i - l * a.n_tiles) * BN;
        const int4 e = __ldg(a.table + 1 + l);
        t.g = e.x, t.m0 = e.y;
        t.rows = (int)min((long long)e.z, a.n - e.y);
    } else if (GELU) {
        const uint32_t column = i / (uint32_t)a.m_tiles;
        t.g = (int)(column / (uint32_t)a.n_tiles);
        t.m0 = (int)(i - column * a.m_tiles) * 2 * BM;
        t.n0 = (int)(column - t.g * a.n_tiles) * BN;
        t.rows = a.B - t.m0;
    } else {
        const uint32_t m = (uint32_t)a.m_tiles, n = (uint32_t)a.n_tiles;
        const uint32_t g = i / (m * n), in = i - g * m * n, band = in / (BAND * m), j = in - band * BAND * m;
        const uint32_t wide = min(BAND, n - band * BAND), r = j / wide;
        t.g = (int)g;
        t.m0 = (int)r * 2 * BM;
        t.n0 = (int)(band * BAND + j - r * wide) * BN;
        t.rows = a.B - t.m0;
    }
    return t;
}
// The row of x and of the output that the tile's row i is, and its plane of their tensor maps.
template <bool EXPERTS>
__device__ __forceinline__ long long row_of(const Tile& t, int i, const Args& a) {
    return EXPERTS ? (long long)t.m0 + i : (long long)(t.m0 + i) * a.G + t.g;
}
template <bool EXPERTS>
__device__ __forceinline__ int plane_of(const Tile& t) {
    return EXPERTS ? 0 : t.g;
}

// The staging is free again: what was written from it before has been read.
__device__ __forceinline__ void staging_free(int lane) {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
}

// 64 bytes of each row of Y from column n on, through the staging: 32 existing rows by
// TMA (which clips what lies outside Y), the last rows of an expert, whose neighbours
// are another's, unaligned rows and those of more than 2^31 bytes by plain stores.  y: the warp's first row in tmY.
template <typename OUT, bool EXPERTS>
__device__ __forceinline__ void save_piece(const float* v, const Args& a, const CUtensorMap* tmY, int y, int plane,
                                           long long row, int n, int rows, int lane, uint32_t stage) {
    constexpr int E = sizeof(OUT);
    staging_free(lane);
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
    if (n >= a.N) return;
    if (a.tma && (!EXPERTS || rows >= 32)) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(tmY, stage, n * E, y, plane);
            bulk_commit_group();
        }
        return;
    }
    char* dst = reinterpret_cast<char*>(a.y) + (row * (long long)a.N + n) * E;
    const size_t pitch = (size_t)a.step * (size_t)a.N * E;
    const int bytes = min(a.N - n, 64) * E;            // the row's rest may be more bytes than fit 32 bits
    if (a.vec)
        store_rows<true, E>(stage, dst, pitch, rows, bytes, lane);
    else
        store_rows<false, E>(stage, dst, pitch, rows, bytes, lane);
}

// 32 columns of this thread's row in 4 bits: 16 bytes of codes; E: the exponent byte.
__device__ __forceinline__ void round_block(const float* v, uint32_t (&w)[4], uint32_t& E) {
    float m[2] = {};
#pragma unroll
    for (int i = 0; i < 32; i += 2) m[i >> 1 & 1] = max3_nan(m[i >> 1 & 1], fabsf(v[i]), fabsf(v[i + 1]));
    E = fp4_exponent(fp4_abs_bits(max3_nan(m[0], m[0], m[1])));
    const uint64_t s = f2_splat(fp4_inv_scale(E));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) f2_unpack(f2_mul(f2_pack(v[8 * c + i], v[8 * c + i + 1]), s), q[i], q[i + 1]);
        w[c] = fp4_pack8(q);
    }
}

// 128 columns of a warp's rows in 4 bits out of the staging, and their exponent bytes
// (of this lane's row).  A thread that stored its own 16 bytes and its byte made every
// store 32 requests of part of a sector: the FFN at B = 2048 took 684 us with that, 595
// once the codes went through shared memory and TMA.
template <bool EXPERTS>
__device__ __forceinline__ void save_codes(const Args& a, const CUtensorMap* tmY, const Tile& tl, int m_warp, long long row,
                                           int n, int rows, uint32_t E, int lane, uint32_t stage) {
    if (!EXPERTS || rows == 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(tmY, stage, n / 2, tl.m0 + m_warp, plane_of<EXPERTS>(tl));
            bulk_commit_group();
        }
    } else {                                             // an expert's last rows: the next ones are another's
        store_rows<true, 1>(stage, reinterpret_cast<char*>(a.o.codes) + row * a.o.ld + n / 2, (size_t)a.o.ld, rows,
                            (a.N - n) / 2, lane);
    }
    if (lane < rows) {
        uint8_t* p = a.o.scales + (row + lane * a.step) * a.o.lds + n / kFp4Block;
        if (n + 128 <= a.N) {                            // lds is a multiple of 16, n of 128
            *reinterpret_cast<uint32_t*>(p) = E;
        } else {
            for (int b = 0; n + kFp4Block * b < a.N; ++b) p[b] = (uint8_t)(E >> (8 * b));
        }
    }
}

// NARROW: chunks of columns that do not exist are left out.
template <int EPI, bool EXPERTS, bool NARROW>
__global__ void __launch_bounds__(THREADS, 1)
fp4_product_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                   const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmY, const Args args) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    const uint32_t sA = base, sB = base + STAGES * A_BYTES;
    const uint32_t sSFA = base + STAGES * STAGE_BYTES, sSFB = sSFA + STAGES * SF_BYTES;
    const uint32_t sEpi = sSFB + STAGES * SFB_BYTES;
    const uint32_t sBias = sEpi + EPI_WARPS * STAGING, sRing = sBias + EPI_WARPS * BIAS_BYTES, bar0 = sRing + 2 * Scales::BYTES;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + x); };
    auto tempty_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 + x); };
    const uint32_t shared_bar = bar0 + 8u * (2 * STAGES + 4);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (shared_bar + 8u - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t unit = blockIdx.x >> 1, nunits = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmS);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 3);           // the even CTA's: its producer, expecting both CTAs' bytes, and both scale warps
            mbar_init(empty_bar(s), 1);          // multicast commit
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(tfull_bar(x), 1);              // multicast commit
            mbar_init(tempty_bar(x), 2 * GROUP_WARPS);   // the even CTA's: the group's warps of both CTAs
        }
        mbar_init(shared_bar, 2 * GROUP_WARPS / 2);  // the even CTA's: the warps that own the shared columns
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
    const uint32_t tiles = EXPERTS ? (uint32_t)__ldg(&args.table[0].x) * (uint32_t)args.n_tiles : args.units;

    if (warp < 4) {
        regs_dec<REGS_OTHER>();
        if (warp == 0) {
            // ------------------------------ TMA producer ------------------------------
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            Tile next{};
            if (unit < tiles) next = tile_of<EXPERTS, EPI == FP4_GELU>(unit, args);
            for (uint32_t i = unit; ok && i < tiles; i += nunits) {
                const Tile tl = next;
                if (i + nunits < tiles) next = tile_of<EXPERTS, EPI == FP4_GELU>(i + nunits, args);
                const int xrow = tl.m0 + BM * (int)rank, wrow = tl.n0 + BN / 2 * (int)rank;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t fb = mapa_shared(full_bar(stage), 0);
                        if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2u * TX_BYTES);
                        tma_load_3d_pair(&tmX, sA + stage * A_BYTES, fb, kb * 128, xrow, plane_of<EXPERTS>(tl));
                        tma_load_3d_pair(&tmW, sB + stage * B_BYTES, fb, kb * 128, wrow, tl.g);
                        tma_load_3d_pair(&tmS, sSFB + stage * SFB_BYTES, fb, kb * (SF_BYTES / 4), tl.n0 / 128, tl.g);
                    }
                    __syncwarp();
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------ MMA issuer --------------------------------
            const uint32_t idesc = idesc_mxf4(2 * BM, BN);
            const uint64_t a_desc = sw128_operand(sA, 16u), b_desc = sw128_operand(sB, 16u);
            const uint64_t sfa_desc = scale_desc(sSFA), sfb_desc = scale_desc(sSFB);
            int stage = 0, acc = 0;
            uint32_t phase = 0, aphase = 0, cphase = 0, slot = 0;
            bool ok = true;
            for (uint32_t i = unit; ok && i < tiles; i += nunits) {
                // this accumulator's last tile is out, and of the other's tile the shared columns
                if (!wait_bounded(tempty_bar(acc), aphase ^ 1u, abort_flag, args.err, args.timeout_ns) ||
                    !wait_bounded(shared_bar, cphase ^ 1u, abort_flag, args.err, args.timeout_ns))
                    break;
                cphase ^= 1u;
                tc_fence_after();
                const uint32_t d = tmem_base + (acc ? ACC1_COL : 0u);
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!wait_bounded(full_bar(stage), phase, abort_flag, args.err, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t sf = tmem_base + SF_COL + SF_COLS * slot;
                        const uint64_t sa = sfa_desc + (uint32_t)(stage * (SF_BYTES >> 4));
                        const uint64_t sb = sfb_desc + (uint32_t)(stage * (SFB_BYTES >> 4));
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            copy_scales<true>(sf + 4u * q, sa + (uint32_t)(q * (QUAD_BYTES >> 4)));
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                copy_scales<true>(sf + 8u + 8u * q + 4u * h, sb + (uint32_t)((2 * h + q) * (QUAD_BYTES >> 4)));
                        }
                        const uint64_t a = a_desc + (uint32_t)(stage * (A_BYTES >> 4));
                        const uint64_t b = b_desc + (uint32_t)(stage * (B_BYTES >> 4));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_mxf4<true>(d, a + 2u * k, b + 2u * k, with_scale_id(idesc, 2u * (k & 1)), sf + 4u * (k >> 1),
                                            sf + 8u + 8u * (k >> 1), (kb | k) != 0 ? 1u : 0u);
                        umma_commit_pair_mc(empty_bar(stage), (uint16_t)0x3);
                    }
                    __syncwarp();
                    slot ^= 1u;
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair_mc(tfull_bar(acc), (uint16_t)0x3);
                __syncwarp();
                acc ^= 1;
                if (acc == 0) aphase ^= 1u;
            }
        } else if (warp >= 2) {
            // ------------------------------ scales of x -------------------------------
            const int groups = (kblocks + 1) / 2;
            Scales sc(sRing + (warp - 2) * Scales::BYTES);
            uint32_t i = unit;                           // of the next step to fetch
            int g = 0;
            Tile tl{};
            auto skip = [&]() {
                if (++g == groups) {
                    g = 0, i += nunits;
                    if (i < tiles) tl = tile_of<EXPERTS, EPI == FP4_GELU>(i, args);
                }
            };
            auto fetch = [&]() {
                if (i >= tiles) return sc.done();
                const int m0 = BM * (int)rank;
                sc.fetch(args.xs + row_of<EXPERTS>(tl, m0, args) * args.xs_ld, args.step * args.xs_ld, tl.rows - m0, g, lane);
                skip();
                if (i < tiles) skip();
            };
            if (i < tiles) {
                tl = tile_of<EXPERTS, EPI == FP4_GELU>(i, args);
                if (warp == 3) skip();
            }
#pragma unroll 1
            for (int d = 0; d < Scales::STEPS; ++d) fetch();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true, mine = warp == 2;
            for (uint32_t j = unit; ok && j < tiles; j += nunits)
                for (int kb = 0; ok && kb < kblocks; kb += 2, mine = !mine) {
                    if (!mine) {
                        stage += min(2, kblocks - kb);
                        if (stage >= STAGES) stage -= STAGES, phase ^= 1u;
                        continue;
                    }
                    sc.take(kb / 2, args.nb, lane);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (kb + h >= kblocks) break;
                        if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                            ok = false;
                            break;
                        }
                        sc.store(sSFA + stage * SF_BYTES, h, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_pair(mapa_shared(full_bar(stage), 0));
                        if (++stage == STAGES) stage = 0, phase ^= 1u;
                    }
                    fetch();
                }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        // ------------------------------ epilogue --------------------------------------
        regs_inc<REGS_EPI>();
        // the group's accumulator; 32 rows, 128 columns
        const int acc = (warp - 4) / GROUP_WARPS, quad = warp & 3, part = ((warp - 4) >> 2) & 1;
        const uint32_t stage = sEpi + (uint32_t)(warp - 4) * STAGING, bias = sBias + (uint32_t)(warp - 4) * BIAS_BYTES;
        // The 64 columns that the other accumulator shares are the last of accumulator 0
        // and the first of 1: their owners read them first.
        const bool owner = part != acc;
        const int first = acc == 0 && part == 1 ? 1 : 0;             // the half of the warp's columns that comes first
        uint32_t phase = 0;
        // the group's next tile and its bias come while this one is worked on
        Tile next{};
        float b[4] = {};
        auto look_ahead = [&](uint32_t i) {
            if (i >= tiles) return;
            next = tile_of<EXPERTS, EPI == FP4_GELU>(i, args);
            if (args.bias) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int c = next.n0 + WARP_COLS * part + 32 * h + lane;
                    b[h] = c < args.N ? __ldg(args.bias + (size_t)next.g * args.N + c) : 0.f;
                }
            }
        };
        look_ahead(unit + acc * nunits);
        for (uint32_t i = unit + acc * nunits; i < tiles; i += 2 * nunits) {
            const Tile tl = next;
            const int m_warp = BM * (int)rank + 32 * quad, n_warp = tl.n0 + WARP_COLS * part;
            const int rows = n_warp < args.N ? min(32, tl.rows - m_warp) : 0;     // this warp's rows that exist (may be negative)
            const long long row = row_of<EXPERTS>(tl, m_warp, args);
            if (!wait_bounded(tfull_bar(acc), phase, abort_flag, args.err, args.timeout_ns)) break;
            phase ^= 1u;
            tc_fence_after();
            uint32_t E = 0;                                  // (4-bit output) exponent bytes of the row's four blocks
            const uint32_t tcol =
                tmem_base + ((uint32_t)(32 * quad) << 16) + (acc ? ACC1_COL : 0u) + (uint32_t)(WARP_COLS * part);
            // 64 floats of the bias, for the two chunks to come
            auto put_bias = [&](int half) {
                if (!args.bias) return;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(bias + 128u * h + 4u * lane), "f"(half ? b[2 + h] : b[h])
                                 : "memory");
            };
            // 32 columns, the warp's chunk c
            auto finish = [&](const uint32_t (&r)[CHUNK], int c) {
                const int n = n_warp + CHUNK * c;
                if (NARROW && n >= args.N) return;
                float v[CHUNK];
#pragma unroll
                for (int k = 0; k < CHUNK; ++k) v[k] = __uint_as_float(r[k]);
                if (args.bias) {
#pragma unroll
                    for (int k = 0; k < CHUNK / 4; ++k) {
                        float4 q;
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w)
                                     : "r"(bias + 128u * (c & 1) + 16u * k));
                        f2_unpack(f2_add(f2_pack(v[4 * k], v[4 * k + 1]), f2_pack(q.x, q.y)), v[4 * k], v[4 * k + 1]);
                        f2_unpack(f2_add(f2_pack(v[4 * k + 2], v[4 * k + 3]), f2_pack(q.z, q.w)), v[4 * k + 2], v[4 * k + 3]);
                    }
                }
                if constexpr (EPI == FP4_OUT_BF16) {
                    save_piece<__nv_bfloat16, EXPERTS>(v, args, &tmY, tl.m0 + m_warp, plane_of<EXPERTS>(tl), row, n, rows,
                                                       lane, stage);
                } else if constexpr (EPI == FP4_OUT_F32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        save_piece<float, EXPERTS>(v + 16 * h, args, &tmY, tl.m0 + m_warp, plane_of<EXPERTS>(tl), row,
                                                   n + 16 * h, rows, lane, stage);
                } else {
                    uint32_t w[4], e;
#pragma unroll
                    for (int k = 0; k < CHUNK; k += 2) fp4_gelu2(v[k], v[k + 1]);
                    round_block(v, w, e);
                    st_shared_v4(staged_at(stage, lane, c), w[0], w[1], w[2], w[3]);
                    E |= e << (8 * c);
                }
            };
            // Two chunks at once, so that the shared columns are free early; the other two
            // come, one by one, while a chunk is worked on: layer 1 at B = 2048 252 us, 262
            // with 64 columns read, worked on and read again.
            uint32_t r0[CHUNK], r1[CHUNK];
            const int c0 = 2 * first, c2 = 2 - c0;
            tmem_ld32_nowait(tcol + CHUNK * c0, r0);
            tmem_ld32_nowait(tcol + CHUNK * (c0 + 1), r1);
            put_bias(first);
            if (EPI == FP4_GELU) staging_free(lane);
            tmem_wait_ld32(r0);
            tmem_wait_ld32(r1);
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && owner) mbar_arrive_pair(mapa_shared(shared_bar, 0));
            if (rows > 0) {                              // (as a loop: 346 us instead of 252, registers in memory)
                finish(r0, c0);
                tmem_ld32_nowait(tcol + CHUNK * c2, r0);
                finish(r1, c0 + 1);
                __syncwarp();
                put_bias(first ^ 1);
                __syncwarp();
                tmem_wait_ld32(r0);
                tmem_ld32_nowait(tcol + CHUNK * (c2 + 1), r1);
                finish(r0, c2);
                tmem_wait_ld32(r1);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_bar(acc), 0));
            if (rows > 0) finish(r1, c2 + 1);
            look_ahead(i + 2 * nunits);
            if (EPI == FP4_GELU && rows > 0) save_codes<EXPERTS>(args, &tmY, tl, m_warp, row, n_warp, rows, E, lane, stage);
            __syncwarp();
        }
        if (lane == 0) bulk_wait_group<0>();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();    // no CTA leaves while its peer may still touch its memory
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <int EPI, bool EXPERTS, bool NARROW>
cudaError_t run(const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& ms, const CUtensorMap& my, const Args& a,
                int num_sms, cudaStream_t s) {
    auto k = fp4_product_kernel<EPI, EXPERTS, NARROW>;
    cudaError_t e = smem_attr_once((const void*)k, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const long long pairs = num_sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (!EXPERTS && a.units < pairs ? a.units : pairs)));
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
    return cudaLaunchKernelEx(&cfg, k, mx, mw, ms, my, a);
}
// Whether chunks that do not exist are looked for: always but with Gelu, whose registers
// the test costs 4% (layer 1 at B = 2048 262 us instead of 252); there from a quarter of
// the chunks on (51,689 rows of 32 to 32 hidden values and back, three of 11 experts: the
// FFN 58 us instead of 73; 800 hidden values, 3 of 28 chunks: 180 instead of 178).
template <int EPI>
cudaError_t run_for(bool experts, const CUtensorMap& mx, const CUtensorMap& mw, const CUtensorMap& ms, const CUtensorMap& my,
                    const Args& a, int num_sms, cudaStream_t s) {
    const long long there = ((long long)a.N + CHUNK - 1) / CHUNK, all = ((long long)a.N + WARP_COLS - 1) / WARP_COLS * (WARP_COLS / CHUNK);
    if constexpr (EPI == FP4_GELU)
        if (4 * (all - there) < all)
            return experts ? run<EPI, true, false>(mx, mw, ms, my, a, num_sms, s) : run<EPI, false, false>(mx, mw, ms, my, a, num_sms, s);
    return experts ? run<EPI, true, true>(mx, mw, ms, my, a, num_sms, s) : run<EPI, false, true>(mx, mw, ms, my, a, num_sms, s);
}

}  // namespace f4

cudaError_t launch_fp4_product(const Fp4Product& p, const Fp8Device& dev, cudaStream_t s) {
    using namespace f4;
    RM_HOST_BOUNDS(p.B >= 1 && p.G >= 1 && p.K >= 1 && p.N >= 1 && p.n >= 1 && fp4_holds(p.x, p.K));
    RM_HOST_BOUNDS(fp8_on(p.w.codes, 16) && fp8_on(p.w.scales, 16) && p.w.lds == fp4_weight_quads(p.K) &&
                   p.w.ld % 16 == 0 && p.w.ld >= 16 * fp4_blocks(p.K) && (!p.bias || fp8_on(p.bias, 16)));
    RM_HOST_BOUNDS(p.epi == FP4_GELU ? p.N % 32 == 0 && fp4_holds(p.o, p.N) : fp8_on(p.y, 16));
    if (fp4_streams(p, dev)) return launch_fp4_stream(p, dev, s);
    Args a{};
    a.B = p.B, a.G = p.G, a.N = p.N;
    a.m_tiles = (p.B + 2 * BM - 1) / (2 * BM);
    a.n_tiles = (p.N + BN - 1) / BN;
    a.kblocks = (p.K + BK - 1) / BK;
    a.nb = (int)fp4_blocks(p.K);
    a.table = p.tiles;
    // (by expert: tiles at most)
    const long long units = (p.tiles ? p.G + p.n / kExpertTile : (long long)p.G * a.m_tiles) * a.n_tiles;
    if (units >= 1ll << 31) return cudaErrorNotSupported;        // more tiles than a device's memory holds outputs for
    a.units = (uint32_t)units;
    a.n = p.n;
    a.step = p.tiles ? 1 : p.G;
    a.xs = p.x.scales, a.xs_ld = p.x.lds;
    a.bias = p.bias;
    a.y = p.y;
    a.vec = p.N % (p.epi == FP4_OUT_F32 ? 4 : 8) == 0;
    a.o = p.o;
    a.err = dev.err;
    a.timeout_ns = dev.timeout_ns;
    const auto u8t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const long long wide = 16ll * a.nb, tiles = (p.N + kFp4TileRows - 1) / kFp4TileRows;
    CUtensorMap mx, mw, ms;
    const bool ok =
        (p.tiles ? fp8_tensor_map(&mx, u8t, p.x.codes, wide, p.n, 1, p.x.ld, p.x.ld, 128, BM)
                 : fp8_tensor_map(&mx, u8t, p.x.codes, wide, p.B, p.G, p.G * p.x.ld, p.x.ld, 128, BM)) &&
        fp8_tensor_map(&mw, u8t, p.w.codes, wide, p.N, p.G, p.w.ld, p.N * p.w.ld, 128, BN / 2) &&
        fp8_tensor_map(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT32, p.w.scales, p.w.lds * (QUAD_BYTES / 4), tiles, p.G,
                       p.w.lds * QUAD_BYTES, tiles * p.w.lds * QUAD_BYTES, SF_BYTES / 4, 2, true);
    // what leaves by TMA, in bytes: 64 of 32 rows of Y or of the codes
    CUtensorMap my = mx;
    const bool gelu = p.epi == FP4_GELU;
    const long long bytes = gelu ? p.N / 2 : p.N * (p.epi == FP4_OUT_F32 ? 4ll : 2ll), pitch = gelu ? p.o.ld : bytes;
    const void* dst = gelu ? p.o.codes : p.y;
    a.tma = a.vec && bytes <= 1ll << 31;
    if (ok && (gelu || a.tma) &&
        !(p.tiles ? fp8_tensor_map(&my, u8t, dst, bytes, p.n, 1, pitch, pitch, 64, 32)
                  : fp8_tensor_map(&my, u8t, dst, bytes, p.B, p.G, p.G * pitch, pitch, 64, 32)))
        return cudaErrorInvalidValue;
    if (!ok) return cudaErrorInvalidValue;
    switch (p.epi) {
        case FP4_OUT_BF16: return run_for<FP4_OUT_BF16>(p.tiles != nullptr, mx, mw, ms, my, a, dev.num_sms, s);
        case FP4_OUT_F32: return run_for<FP4_OUT_F32>(p.tiles != nullptr, mx, mw, ms, my, a, dev.num_sms, s);
        case FP4_GELU: return run_for<FP4_GELU>(p.tiles != nullptr, mx, mw, ms, my, a, dev.num_sms, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace rm
