// Weight gradient of a per-token linear layer from its input kept in 8 bits,
//   dW[t][k][n] = sum_b x[b][t][k] dY[b][t][n]   (dY bf16),
// on the 5th-generation tensor cores.  The scales of x belong to the summed
// index (one per sample and 128 values of k), so they cannot be applied by a
// block-scaled MMA, whose scales run along the sum in blocks: x's codes are
// restored on the way, in shared memory.  A code times a power of two is exact
// in bf16, so the product is the bf16 product of the restored activation and
// dY, without that activation ever being written to memory: x costs one byte a
// value, and no pass of its own.
//
// Kernel: one persistent pair of CTAs per 256 (k) x 256 (n) tile of one token;
// per 64 samples each CTA holds 128 of x's columns and 128 of dY's.
//   warp 0        TMA producer of dY (MN-major: boxes of 64 columns x 64 samples)
//   warp 1        MMA issuer (the even CTA's): kind::f16 on bf16, M = N = 256
//   warp 2        TMA producer of x's codes (64 samples x 128 bytes)
//   warps 4-11    epilogue
//   warps 20-23   db, the column sums of dY, in one tile of each column of tiles:
//                 from dY's operand tile in shared memory once the MMA is done with
//                 it, so dY is not read again
//   warp 3        x's exponent bytes into shared memory, eight k-blocks' loads
//                 at a time so that their latency is paid once in eight
//   warps 12-19   restore codes to bf16: MN-major operand rows are samples, so
//                 16 codes of a row become two 16-byte pieces of the same row.
//                 Two codes at a time: the bits of e4m3, moved to bf16's
//                 exponent and mantissa, are the code times 2^-120 (also for
//                 subnormal codes), so one packed product by 2^120 times the
//                 scale restores it: 4 instructions for two codes
// db's sums cost a hop on the operand ring, so only the k-blocks that are summed
// take it (all of them did at first: 844 us against 816 at the size below, in f32).
//
// Measured, T = 32, K = 1536, N = 6144, dW and db: B = 2048 812 us in f32 (1523
// TFLOP/s) and 783 us in bf16, B = 1024 472 and 422 us; B = 8, where a tile is one
// k-block and the time is dW's, 207 us (5.8 TB/s) and 109 us (5.5 TB/s).  Bound at
// large B by the tensor cores under the power limit and the restorers beside them
// (shared memory), at small B by dW's stores.
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error
// word and all roles unwind.
#include <cudaTypedefs.h>

#include "rm_fp8.cuh"
#include "rm_fp8_tc.cuh"

namespace rm {
namespace f8w {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int RAW_BYTES = BK * BM;           // 64 samples x 128 codes
constexpr int A_BYTES = BK * BM * 2;         // the same in bf16: two boxes of 64 columns x 64 samples
constexpr int B_BYTES = BK * (BN / 2) * 2;   // dY: two boxes of 64 columns x 64 samples
constexpr int BOX_BYTES = 64 * BK * 2;
constexpr int STAGES = 4, RAWS = 8;
constexpr int EPI_WARPS = 8, CONV_WARPS = 8;
constexpr int CONV_GROUP = 2;                // restoring warps per k-block
constexpr int GROUPS = CONV_WARPS / CONV_GROUP;
constexpr int AHEAD = 8;                     // k-blocks whose exponent bytes are loaded together
// Float32 gradients of more samples are summed in chunks of this many: a chunk's
// sum leaves the tensor cores' accumulator (which truncates each addition) and
// is added to dW in memory with rounding to nearest.
constexpr int CHUNK = 2048;
constexpr int STAGING = 4096;
constexpr int SUM_WARPS = 4;                 // 32 columns of dY each
constexpr int SUM_WARP0 = 4 + EPI_WARPS + CONV_WARPS;
constexpr int THREADS = 32 * (SUM_WARP0 + SUM_WARPS);
constexpr int SMEM_BYTES = 1024 + STAGES * (A_BYTES + B_BYTES) + RAWS * (RAW_BYTES + BK) + EPI_WARPS * STAGING + 320;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(GROUPS <= RAWS && GROUPS <= STAGES, "a k-block per group of restorers");

struct Args {
    int B, T, K, N;
    int m_tiles, n_tiles, kblocks;
    int chunks, chunk_blocks;            // the sum over samples: chunks of that many k-blocks
    long long tiles;
    const uint8_t* xs;
    long long xs_ld;
    void* db;                            // [T][N] or null
    int* err;
    unsigned long long timeout_ns;
};

struct Tile {
    int t, m0, n0;
    bool sums;                           // adds up dY's columns: one tile of each column of tiles
};
__device__ __forceinline__ Tile tile_of(long long i, const Args& a) {
    const int per = a.m_tiles * a.n_tiles;
    Tile r;
    r.t = (int)(i / per);
    const int rem = (int)(i - (long long)r.t * per), nb = rem / a.m_tiles;
    r.m0 = (rem - nb * a.m_tiles) * 2 * BM;
    r.n0 = nb * BN;
    // not always the first: tiles go round the CTA pairs, and the pairs' number may share
    // a factor with m_tiles, which would leave all the sums to a few of them
    r.sums = rem - nb * a.m_tiles == (int)((unsigned)(r.t + nb) % (unsigned)a.m_tiles);
    return r;
}

// kind::f16: D f32, A and B bf16, both MN-major, N >> 3, M >> 4.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(BN >> 3) << 17) |
                            ((uint32_t)(2 * BM >> 4) << 24);

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two codes (bytes of w) to bf16 times 2^-120: the selector spreads them to
// halves with their sign bits repeated above (prmt's sign mode), which leaves
// the sign at bit 15 and the magnitude's seven bits at bit 4 after the shift.
__device__ __forceinline__ uint32_t spread2(uint32_t w, uint32_t selector) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "r"(selector));
    return (r << 4) & 0x87f087f0u;
}

// 16 codes to 16 bf16 of code * 2^(E - 127): exact where bf16 is normal, else
// rounded once.  restore16 is for blocks up to 57344 (E <= 134: 2^120 2^(E - 127)
// is a bf16) without NaN codes; restore16_any takes the rest.
__device__ __forceinline__ bool plain16(const uint4& q, uint32_t E) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t nan = 0;                                  // codes of magnitude 0x7f
#pragma unroll
    for (int i = 0; i < 4; ++i) nan |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
    return E <= 134u && (nan & 0x80808080u) == 0u;
}
__device__ __forceinline__ void restore16(const uint4& q, uint32_t E, uint32_t (&o)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const uint32_t h = (E + 120u) << 7, s = h | (h << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = mul_bf16x2(spread2(w[i], 0x9180u), s);
        o[2 * i + 1] = mul_bf16x2(spread2(w[i], 0xb3a2u), s);
    }
}
__device__ __noinline__ void restore16_any(const uint4& q, uint32_t E, uint32_t (&o)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const uint32_t h = E == 255u ? 0x7fc0u : E == 0u ? 0x0040u : E << 7, s = h | (h << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {                      // in two steps, the first exact
        o[2 * i] = mul_bf16x2(mul_bf16x2(spread2(w[i], 0x9180u), 0x7b807b80u), s);
        o[2 * i + 1] = mul_bf16x2(mul_bf16x2(spread2(w[i], 0xb3a2u), 0x7b807b80u), s);
        const uint32_t m = ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        o[2 * i] |= (m & 0x80u ? 0x7fffu : 0u) | (m & 0x8000u ? 0x7fff0000u : 0u);
        o[2 * i + 1] |= (m & 0x800000u ? 0x7fffu : 0u) | (m & 0x80000000u ? 0x7fff0000u : 0u);
    }
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Tiled add of float32 shared -> global (bulk async group).
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

template <bool F32>
__global__ void __launch_bounds__(THREADS, 1)
fp8_wgrad_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY,
                 const __grid_constant__ CUtensorMap tmW, const Args args) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    const uint32_t sA = base, sB = sA + STAGES * A_BYTES, sRaw = sB + STAGES * B_BYTES;
    const uint32_t sEpi = sRaw + RAWS * RAW_BYTES, sExp = sEpi + EPI_WARPS * STAGING;
    const uint32_t bar0 = sExp + RAWS * BK;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto rfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto rempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + RAWS + s); };
    auto tfull_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * RAWS + x); };
    auto tempty_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * RAWS + 2 + x); };
    auto summed_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 2 * RAWS + 4 + s); };
    auto sready_bar = [&](int s) { return bar0 + 8u * (3 * STAGES + 2 * RAWS + 4 + s); };
    uint32_t* tmem_holder =
        reinterpret_cast<uint32_t*>(base_ptr + (bar0 - base) + 8 * (4 * STAGES + 2 * RAWS + 4));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const long long unit = blockIdx.x >> 1, nunits = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmY);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1 + 2 * CONV_GROUP);   // the even CTA's: dY's bytes of both CTAs, both CTAs' restorers
            mbar_init(empty_bar(s), 1);                   // multicast commit
            mbar_init(sready_bar(s), 1);                  // the same, for k-blocks of tiles that are summed
            mbar_init(summed_bar(s), SUM_WARPS);          // ... and these have been summed
        }
        for (int s = 0; s < RAWS; ++s) {
            mbar_init(rfull_bar(s), 2);                   // x's bytes, its exponents
            mbar_init(rempty_bar(s), CONV_GROUP);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(tfull_bar(x), 1);                   // multicast commit
            mbar_init(tempty_bar(x), 2 * EPI_WARPS);      // the even CTA's: every epilogue warp of both CTAs
        }
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

    if (warp == 0) {
        // ------------------------------ dY producer -------------------------------
        int stage = 0;
        uint32_t phase = 0;
        uint32_t held = 0, sphase = 0;         // per stage: holds a k-block to be summed; its barrier's phase
        bool ok = true;
        for (long long i = unit; ok && i < args.tiles; i += nunits) {
            const Tile tl = tile_of(i, args);
            const int col = tl.n0 + BN / 2 * (int)rank;
            for (int kb = 0; kb < kblocks; ++kb) {
                const uint32_t bit = 1u << stage;
                const bool summed = (held & bit) != 0;
                if (!wait_bounded(summed ? summed_bar(stage) : empty_bar(stage),
                                  summed ? (uint32_t)((sphase & bit) != 0) : phase ^ 1u, abort_flag, args.err,
                                  args.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (summed) sphase ^= bit;
                held = args.db && tl.sums ? held | bit : held & ~bit;
                if (elect_one()) {
                    const uint32_t fb = mapa_shared(full_bar(stage), 0);
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2u * B_BYTES);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        tma_load_3d_pair(&tmY, sB + stage * B_BYTES + j * BOX_BYTES, fb, col + 64 * j, kb * BK, tl.t);
                }
                __syncwarp();
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
    } else if (warp == 2) {
        // ------------------------------ x producer --------------------------------
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (long long i = unit; ok && i < args.tiles; i += nunits) {
            const Tile tl = tile_of(i, args);
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!wait_bounded(rempty_bar(slot), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(rfull_bar(slot), RAW_BYTES);
                    tma_load_3d(&tmX, sRaw + slot * RAW_BYTES, rfull_bar(slot), tl.m0 + BM * (int)rank, kb * BK, tl.t);
                }
                __syncwarp();
                if (++slot == RAWS) slot = 0, phase ^= 1u;
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------ MMA issuer --------------------------------
        const uint64_t a_desc = sw128_operand(sA, BOX_BYTES), b_desc = sw128_operand(sB, BOX_BYTES);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (long long i = unit; ok && i < args.tiles; i += nunits) {
            const bool sums = args.db && tile_of(i, args).sums;
            int in_chunk = 0;
            for (int kb = 0; kb < kblocks; ++kb) {
                if (in_chunk == 0 &&
                    !wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t d = tmem_base + (uint32_t)(acc * BN);
                if (!wait_bounded(full_bar(stage), phase, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t a = a_desc + (uint32_t)(stage * (A_BYTES >> 4));
                    const uint64_t b = b_desc + (uint32_t)(stage * (B_BYTES >> 4));
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)        // 16 samples: 16 rows of 128 bytes
                        umma_f16_pair(d, a + 128u * k, b + 128u * k, kIdesc, (in_chunk | k) != 0 ? 1u : 0u);
                    umma_commit_pair_mc(empty_bar(stage), (uint16_t)0x3);
                    if (sums) umma_commit_pair_mc(sready_bar(stage), (uint16_t)0x3);
                }
                __syncwarp();
                if (++stage == STAGES) stage = 0, phase ^= 1u;
                if (++in_chunk == args.chunk_blocks || kb + 1 == kblocks) {
                    if (elect_one()) umma_commit_pair_mc(tfull_bar(acc), (uint16_t)0x3);
                    __syncwarp();
                    in_chunk = 0;
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
        }
    } else if (warp == 3) {
        // ------------------------------ exponents ---------------------------------
        // AHEAD k-blocks at a time, across the ends of tiles: with one k-block per tile
        // (few samples) each tile would otherwise wait for a load of its own.
        int slot = 0, kb = 0, k0 = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint8_t* sp = args.xs;
        const size_t step = (size_t)args.T * (size_t)args.xs_ld;
        for (long long i = unit; ok && i < args.tiles;) {
            uint32_t E[AHEAD][2];
            int n = 0;
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                if (i < args.tiles) {
                    if (kb == 0) {
                        const Tile tl = tile_of(i, args);
                        k0 = tl.m0 + BM * (int)rank;
                        sp = args.xs + (size_t)tl.t * (size_t)args.xs_ld + k0 / kFp8Block;
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int b = kb * BK + 32 * j + lane;
                        E[q][j] = b < args.B && k0 < args.K ? __ldg(sp + (size_t)b * step) : 127u;
                    }
                    if (++kb == kblocks) kb = 0, i += nunits;
                    n = q + 1;
                }
            }
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                if (ok && q < n) {
                    ok = wait_bounded(rempty_bar(slot), phase ^ 1u, abort_flag, args.err, args.timeout_ns);
                    if (ok) {
                        st_shared_u8(sExp + BK * slot + lane, E[q][0]);
                        st_shared_u8(sExp + BK * slot + 32 + lane, E[q][1]);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(rfull_bar(slot));
                        if (++slot == RAWS) slot = 0, phase ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= SUM_WARP0) {
        // ------------------------------ bias gradient -----------------------------
        // Lane: 8 columns (16 bytes) of every eighth row.  Eight lanes read four chunks of
        // rows r and r + 4, whose swizzles have no bank in common.  Only the k-blocks of
        // tiles that are summed pass through here on their way back to the dY producer,
        // by barriers of their own, whose phases count those k-blocks alone.
        const int box = (warp - SUM_WARP0) >> 1, c = (lane & 3) + 4 * ((warp - SUM_WARP0) & 1);
        const int r0 = (lane >> 3) + (lane & 4);
        int stage = 0;
        uint32_t phase = 0;                            // per stage
        bool ok = true;
        for (long long i = unit; args.db && ok && i < args.tiles; i += nunits) {
            const Tile tl = tile_of(i, args);
            if (!tl.sums) {
                stage = (stage + kblocks) % STAGES;
                continue;
            }
            // float32 sums are joined from sums of a chunk, as dW's are: in one running sum a
            // value that is constant over the samples would be rounded the same way each time
            float total[8] = {}, sum[8] = {};
            int in_chunk = 0;
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!wait_bounded(sready_bar(stage), (phase >> stage) & 1u, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                phase ^= 1u << stage;
                const uint32_t src = sB + stage * B_BYTES + box * BOX_BYTES;
#pragma unroll
                for (int r = r0; r < BK; r += 8) {
                    const uint4 q = ld_shared_u4(src + 128u * r + 16u * (uint32_t)(c ^ (r & 7)));
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sum[2 * j] += __uint_as_float(w[j] << 16);
                        sum[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(summed_bar(stage));
                if (++stage == STAGES) stage = 0;
                if (++in_chunk == args.chunk_blocks) {
                    in_chunk = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) total[j] += sum[j], sum[j] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum[j] += total[j];
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 4);
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
                sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
            }
            const int n = tl.n0 + BN / 2 * (int)rank + 64 * box + 8 * c;
            if (ok && lane < 4 && n < args.N) {       // N is a multiple of 8
                const size_t at = (size_t)tl.t * args.N + n;
                if (F32) {
                    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(args.db) + at);
                    o[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
                    o[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
                } else {
                    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(args.db) + at) =
                        make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]),
                                   pack_bf16x2(sum[4], sum[5]), pack_bf16x2(sum[6], sum[7]));
                }
            }
        }
    } else if (warp >= 12) {
        // ------------------------------ restorers ---------------------------------
        // Four groups of two warps, each with every fourth k-block, so that one's
        // latencies (barriers, shared memory, the fence) pass while others work.
        // Lane's 16-byte chunks: column chunk c of eight of its warp's 32 rows.  The two
        // rows that a group of eight lanes reads at a time differ by 5 in their low
        // three bits, which keeps both the reads (chunk c of row r at c ^ (r % 8)) and
        // the writes (pieces 2 (c % 4), + 1 at ^ (r % 8)) free of bank conflicts.
        const uint32_t cw = (uint32_t)(warp - 12) % CONV_GROUP, group = (uint32_t)(warp - 12) / CONV_GROUP;
        const uint32_t c = (lane & 3) | ((lane >> 1) & 4), p = 2u * (c & 3u);
        const uint32_t flip = (lane & 4) ? 5 : 0, rep0 = lane >> 4;
        uint32_t slot = group;
        uint32_t rphase = 0;
        int stage = (int)group;                      // of the group's next k-block
        uint32_t phase = 0;
        long long left = ((args.tiles - 1 - unit) / nunits + 1) * kblocks - group;   // unit < tiles: the grid's size
        for (; left > 0; left -= GROUPS) {
            if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns) ||
                !wait_bounded(rfull_bar(slot), rphase, abort_flag, args.err, args.timeout_ns))
                break;
            const uint32_t src = sRaw + slot * RAW_BYTES, exps = sExp + BK * slot;
            const uint32_t dst = sA + stage * A_BYTES + (c >> 2) * BOX_BYTES;
            // all chunks are loaded first and restored without a branch between them
            constexpr int CH = BK / CONV_GROUP / 4;
            uint4 q[CH];
            uint32_t E[CH];
            bool plain = true;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const uint32_t x7 = (rep0 | ((j & 1u) << 1)) ^ flip, r = BK / CONV_GROUP * cw + 8u * (j >> 1) + x7;
                q[j] = ld_shared_u4(src + 128u * r + 16u * (c ^ x7));
                E[j] = ld_shared_u8(exps + r);
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) plain = plain && plain16(q[j], E[j]);
            auto put = [&](int j, const uint32_t (&o)[8]) {
                const uint32_t x7 = (rep0 | ((j & 1u) << 1)) ^ flip, r = BK / CONV_GROUP * cw + 8u * (j >> 1) + x7;
                st_shared_v4(dst + 128u * r + 16u * (p ^ x7), o[0], o[1], o[2], o[3]);
                st_shared_v4(dst + 128u * r + 16u * ((p + 1u) ^ x7), o[4], o[5], o[6], o[7]);
            };
            if (plain) {
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    uint32_t o[8];
                    restore16(q[j], E[j], o);
                    put(j, o);
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < CH; ++j) {
                    uint32_t o[8];
                    const uint32_t x7 = (rep0 | ((j & 1u) << 1)) ^ flip, r = BK / CONV_GROUP * cw + 8u * (j >> 1) + x7;
                    restore16_any(ld_shared_u4(src + 128u * r + 16u * (c ^ x7)), ld_shared_u8(exps + r), o);
                    put(j, o);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_pair(mapa_shared(full_bar(stage), 0));
                mbar_arrive(rempty_bar(slot));
            }
            stage += GROUPS;
            if (stage >= STAGES) stage -= STAGES, phase ^= 1u;
            slot += GROUPS;
            if (slot >= RAWS) slot -= RAWS, rphase ^= 1u;
        }
    } else if (warp >= 4) {
        // ------------------------------ epilogue ----------------------------------
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t stage = sEpi + (uint32_t)(warp - 4) * STAGING;
        constexpr int PIECE = F32 ? 32 : 64;                 // columns of 128 bytes
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (long long i = unit; ok && i < args.tiles; i += nunits) {
          const Tile tl = tile_of(i, args);
          for (int chunk = 0; chunk < args.chunks; ++chunk) {
            const int m = tl.m0 + BM * (int)rank + 32 * quad, n = tl.n0 + 128 * half;
            if (!wait_bounded(tfull_bar(acc), acc_phase, abort_flag, args.err, args.timeout_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t tcol = tmem_base + ((uint32_t)(32 * quad) << 16) + (uint32_t)(acc * BN) + 128u * half;
#pragma unroll
            for (int h = 0; h < 128 / PIECE; ++h) {
#pragma unroll 1                              // unrolled, both halves' registers are live and spill
                for (int q = 0; q < PIECE / 32; ++q) {
                    uint32_t r[32];
                    tmem_ld32_nowait(tcol + PIECE * h + 32 * q, r);
                    tmem_wait_ld();
                    if (q == 0) {
                        if (lane == 0) {
                            if (F32 && chunk > 0)
                                bulk_wait_group<0>();        // the chunk before is in memory
                            else
                                bulk_wait_group_read<0>();
                        }
                        __syncwarp();
                    }
                    constexpr int PER = F32 ? 4 : 8;         // columns in 16 bytes
#pragma unroll
                    for (int p = 0; p < 32 / PER; ++p) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = F32 ? r[4 * p + j]
                                       : pack_bf16x2(__uint_as_float(r[(8 * p + 2 * j) % 32]),
                                                     __uint_as_float(r[(8 * p + 2 * j + 1) % 32]));
                        const uint32_t c = (uint32_t)(p + q * (32 / PER));
                        st_shared_v4(stage + 128u * lane + 16u * (c ^ (lane & 7)), w[0], w[1], w[2], w[3]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (m < args.K && n + PIECE * h < args.N) {
                        if (F32 && chunk > 0)
                            tma_add_3d(&tmW, stage, n + PIECE * h, m, tl.t);
                        else
                            tma_store_3d(&tmW, stage, n + PIECE * h, m, tl.t);
                    }
                    bulk_commit_group();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_bar(acc), 0));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
        }
        if (lane == 0) bulk_wait_group<0>();                 // this warp's tensor stores have landed
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();    // no CTA leaves while its peer may still touch its memory
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <bool F32>
cudaError_t run(const CUtensorMap& mx, const CUtensorMap& my, const CUtensorMap& mw, const Args& a, int num_sms,
                cudaStream_t s) {
    auto k = fp8_wgrad_kernel<F32>;
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
    e = cudaLaunchKernelEx(&cfg, k, mx, my, mw, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace f8w

cudaError_t launch_fp8_wgrad(const Fp8View& x, const void* dY, void* dW, void* db, bool f32, int B, int T, int K, int N,
                             const Fp8Device& dev, cudaStream_t s) {
    using namespace f8w;
    RM_HOST_BOUNDS(B >= 1 && T >= 1 && K >= 1 && N >= 1 && N % 8 == 0 && fp8_holds(x, K) && !x.e5m2);
    RM_HOST_BOUNDS(fp8_on(dY, 16) && fp8_on(dW, 16) && (!db || fp8_on(db, 16)));
    Args a{};
    a.B = B, a.T = T, a.K = K, a.N = N;
    a.m_tiles = (K + 2 * BM - 1) / (2 * BM);
    a.n_tiles = (N + BN - 1) / BN;
    a.kblocks = (B + BK - 1) / BK;
    a.tiles = (long long)T * a.m_tiles * a.n_tiles;
    a.chunk_blocks = f32 ? CHUNK / BK : a.kblocks;
    a.chunks = (a.kblocks + a.chunk_blocks - 1) / a.chunk_blocks;
    a.xs = x.scales, a.xs_ld = x.lds;
    a.db = db;
    a.err = dev.err;
    a.timeout_ns = dev.timeout_ns;
    CUtensorMap mx, my, mw;
    if (!fp8_tensor_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x.codes, K, B, T, T * x.ld, x.ld, BM, BK) ||
        !fp8_tensor_map(&my, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dY, N, B, T, 2ll * T * N, 2ll * N, 64, BK) ||
        !fp8_tensor_map(&mw, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dW, N, K, T,
                        (f32 ? 4ll : 2ll) * N, (f32 ? 4ll : 2ll) * K * N, f32 ? 32 : 64, 32))
        return cudaErrorInvalidValue;
    return f32 ? run<true>(mx, my, mw, a, dev.num_sms, s) : run<false>(mx, my, mw, a, dev.num_sms, s);
}

}  // namespace rm
