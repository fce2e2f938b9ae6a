// Per-token products of 8-bit operands for few samples: the same product as
// rm_fp8_gemm.cu with W's columns as the rows of the MMA, so that a token's
// weights are streamed once and nothing is computed for samples that are not
// there.
//   acc[n][b] = sum_k W[t][k][n] x[b][t][k],  128 columns n x NB samples a tile
// Bound by memory: W is read once (T K N bytes), at one sample 99% of the
// traffic, so the kernel is a deep pipeline of weight tiles: one persistent CTA
// per SM, 16 KB of W (128 x 128 codes) and NB rows of x per k-block and stage,
// 152 x 180 KB in flight.
//   warp 0       TMA producer of W ([K][N]: MN-major; [N][K]: K-major)
//   warp 1       MMA issuer (tcgen05.mma kind::mxf8f6f4, M = 128, N = NB, one CTA)
//   warp 2       scales (as in rm_fp8_gemm.cu: words of four k-blocks' exponents)
//   warp 3       TMA producer of x
//   warps 4-7 (to 11 for more than 16 samples, to 19 for more than 64)  epilogue: a
//                thread owns one column n of 16 or 32 samples; an 8-bit output's
//                block of 128 columns is four warps' threads, whose largest values
//                meet in a warp maximum and four words of shared memory; one thread
//                per sample then makes the scale that the others read
// A CTA walks all of its tile's K by itself, so where the tiles are few, most SMs
// would idle: then 2 or 4 CTAs (a cluster) each take a part of K.  The first one's
// epilogue adds the others' sums, which they store straight from registers into
// what its ring leaves free of its shared memory; always in the same order.
// More than 128 samples come here, as several tiles of samples, only where all tiles
// fit on the SMs at once.
// Measured (within a graph): T = 32, K = 1536, N = 6144, bf16 out, one sample 48.3
// us = 6.3 TB/s of W, 64 samples 54 us, 128 samples 61 us; K = 6144, N = 1536 (384
// tiles, 2.5 rounds of the SMs) 53.5, 55.6 and 59.5 us.  Few tiles are bound by
// latency: T = 8, K = 512, N = 2048 3.2 us, K = 2048, N = 512 (32 tiles) 4.6 us, 7.1
// without sharing K.
// The kernel is launched while its predecessor may still run.  Where that
// predecessor is one of this library's own launches of the same call, W was in
// memory before it began, and warp 0 starts on it at once; everything else
// waits for the predecessor's end.
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error
// word and all roles unwind.
#include <cudaTypedefs.h>

#include <type_traits>

#include "rm_fp8.cuh"
#include "rm_fp8_tc.cuh"

namespace rm {
namespace f8s {

constexpr int BM = 128, BK = 128;
constexpr int SAMPLES_MAX = 128;             // of a tile
constexpr int W_BYTES = BM * BK;
constexpr int SF_SLOTS = 4, SF_BYTES = 1024;
// Where as many clusters are resident at once as there are tiles, 2 or 4 CTAs share each
// tile's K.  Of clusters of four 36 are resident (not 38, a quarter of the SMs): K = 2048,
// 8 samples 4.7 us for 36 tiles, 8.0 for 37 with a second round of them, 5.2 with clusters
// of two.  Only 2 for more than 32 samples, whose sums (32 KB from each CTA into one) take
// longer than the shorter K saves: T = 8, K = 2048, N = 512, 64 samples 6.9 us with 4, 6.5
// with 2, 7.6 with 1; 16 samples 4.6 with 4, 7.1 with 1.
constexpr int MAX_SPLIT = 4, MAX_SPLIT_64 = 2;

// Four words to another CTA's shared memory, counted there by its barrier.
__device__ __forceinline__ void st_async_v4(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
// A phase already seen to be complete, looked at once more so that what other CTAs
// of the cluster stored for it is seen too.
__device__ __forceinline__ void mbar_acquire_cluster(uint32_t bar, uint32_t parity) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar), "r"(parity)
        : "memory");
}

template <int NB>
struct Cfg {
    static constexpr int X_BYTES = NB * BK;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int FIT = (200 * 1024) / STAGE_BYTES;
    static constexpr int STAGES = FIT < 12 ? FIT : 12;
    // FFN of T = 8, D = 512, F = 2048: 32 samples 12.4 us with 4 warps, 11.7 with 8;
    // 64 samples 14.25 with 8 or 16, but T = 32, D = 1536, F = 6144 113 with 8, 116 with 16
    static constexpr int EPI_WARPS = NB == 16 ? 4 : NB == 128 ? 16 : 8;
    static constexpr int TMEM_COLS = NB == 128 ? 512 : 256, SF_COL = NB == 128 ? 256 : 192;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int SAMPLES = NB / (EPI_WARPS / 4);            // per epilogue thread
    static constexpr int PART_BYTES = BM * NB * 4;                  // one CTA's partial sums of a split tile
    static constexpr int RED_BYTES = 2 * (4 + 1) * NB * 4;          // [output][warp of the block, then the scale][sample]
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + SF_SLOTS * SF_BYTES + RED_BYTES + 512;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    static_assert(((NB > 32 ? MAX_SPLIT_64 : MAX_SPLIT) - 1) * PART_BYTES <= STAGES * STAGE_BYTES / 2,
                  "half of the ring remains when K is split");
    static_assert(2 * NB <= SF_COL, "two accumulators below the scales");
};

enum Epi { EPI_BF16, EPI_F32, EPI_GELU, EPI_GELU_KEEP, EPI_DGELU };

struct Args {
    int B, T, K, N;
    int n_tiles, m_tiles, kblocks, tiles;
    int split, groups;                   // CTAs (a cluster) that share a tile's K; groups of four k-blocks for each
    int stages;                          // of the ring; what a split's partial sums take is not part of it
    const uint8_t* xs;
    long long xs_ld;
    const uint8_t* ws;
    long long ws_ld;
    int w_rows;
    uint32_t x_format;
    bool early;                          // W may be read before the predecessor's end
    const float* bias;
    void* y;
    Fp8View o0, o1;
    int* err;
    unsigned long long timeout_ns;
};

struct Tile {
    int t, n0, b0;
};
// Sample tiles fastest: those that share a weight tile run side by side.
__device__ __forceinline__ Tile tile_of(int i, const Args& a) {
    Tile r{0, 0, 0};
    if (a.m_tiles > 1) {
        const int q = i / a.m_tiles;
        r.b0 = (i - q * a.m_tiles) * SAMPLES_MAX;
        i = q;
    }
    r.t = i / a.n_tiles;
    r.n0 = (i - r.t * a.n_tiles) * BM;
    return r;
}

template <int EPI, bool TRANS, int NB>
__global__ void __launch_bounds__(Cfg<NB>::THREADS, 1)
fp8_stream_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Args args) {
    using C = Cfg<NB>;
    constexpr int STAGES = C::STAGES, EPI_WARPS = C::EPI_WARPS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    const int stages = args.stages;
    const uint32_t sW = base, sX = sW + stages * W_BYTES, sSF = base + STAGES * C::STAGE_BYTES;
    const uint32_t sPart = sX + stages * C::X_BYTES;        // [rank - 1][sample / 4][column][sample % 4] float
    uint32_t* red = reinterpret_cast<uint32_t*>(base_ptr + (sSF - base) + SF_SLOTS * SF_BYTES);
    const uint32_t bar0 = sSF + SF_SLOTS * SF_BYTES + C::RED_BYTES;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + SF_SLOTS + s); };
    auto tfull_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + x); };
    auto tempty_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + 2 + x); };
    const uint32_t meet_bar = bar0 + 8u * (2 * STAGES + 2 * SF_SLOTS + 4);
    const uint32_t part_bar = meet_bar + 8u * (EPI_WARPS / 4);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (part_bar + 8u - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 2);            // W's bytes, x's bytes
            mbar_init(empty_bar(s), 1);
        }
        for (int s = 0; s < SF_SLOTS; ++s) {
            mbar_init(sfull_bar(s), 1);
            mbar_init(sempty_bar(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(tfull_bar(x), 1);
            mbar_init(tempty_bar(x), EPI_WARPS);
        }
        for (int g = 0; g < EPI_WARPS / 4; ++g) mbar_init(meet_bar + 8u * g, 4);
        mbar_init(part_bar, 1);                   // the other CTAs' partial sums
        *abort_flag = 0;
        fence_mbar_init();
        if (args.split > 1 && cluster_ctarank() == 0)
            mbar_arrive_expect_tx(part_bar, (uint32_t)(args.split - 1) * C::PART_BYTES);
    }
    if (warp == 4) {
        tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (args.split > 1) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
    // this CTA's tiles, and its k-blocks of each
    const int rank = args.split > 1 ? (int)cluster_ctarank() : 0;
    const int unit = (int)blockIdx.x / args.split, units = (int)gridDim.x / args.split;
    const int kb0 = 4 * args.groups * rank;
    const int kb1 = min(kb0 + 4 * args.groups, args.kblocks);
    if (!(args.early && warp == 0)) {
        pdl_wait();
        pdl_launch_next();
    }

    if (warp == 0 || warp == 3) {
        // ------------------------------ TMA producers -----------------------------
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = unit; ok && i < args.tiles; i += units) {
            const Tile tl = tile_of(i, args);
            const int t = tl.t, n0 = tl.n0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (warp == 0) {
                        mbar_arrive_expect_tx(full_bar(stage), W_BYTES);
                        if (TRANS)
                            tma_load_3d(&tmW, sW + stage * W_BYTES, full_bar(stage), kb * BK, n0, t);
                        else
                            tma_load_3d(&tmW, sW + stage * W_BYTES, full_bar(stage), n0, kb * BK, t);
                    } else {
                        mbar_arrive_expect_tx(full_bar(stage), C::X_BYTES);
                        tma_load_3d(&tmX, sX + stage * C::X_BYTES, full_bar(stage), kb * BK, tl.b0, t);
                    }
                }
                __syncwarp();
                if (++stage == stages) stage = 0, phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer --------------------------------
        const uint32_t idesc = idesc_mxf8(BM, NB, !TRANS, false) | (args.x_format << 10);
        constexpr uint32_t a_step = TRANS ? 32u : 32u * 128u;
        const uint64_t a_desc = sw128_operand(sW, TRANS ? 16u : (uint32_t)W_BYTES), b_desc = sw128_operand(sX, 16u);
        int stage = 0, slot = 0, acc = 0;
        uint32_t phase = 0, sphase = 0, acc_phase = 0;
        bool ok = true;
        for (int i = unit; ok && i < args.tiles; i += units) {
            if (!wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag, args.err, args.timeout_ns)) break;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc * NB);
            for (int kb = kb0; kb < kb1; ++kb) {
                const uint32_t sf = tmem_base + C::SF_COL + 8u * slot;
                if ((kb & 3) == 0) {
                    if (!wait_bounded(sfull_bar(slot), sphase, abort_flag, args.err, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        copy_scales<false>(sf, scale_desc(sSF + slot * SF_BYTES));
                        copy_scales<false>(sf + 4, scale_desc(sSF + slot * SF_BYTES + 512));
                    }
                    __syncwarp();
                }
                if (!wait_bounded(full_bar(stage), phase, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const bool last = (kb & 3) == 3 || kb + 1 == kb1;
                if (elect_one()) {
                    const uint32_t id = with_scale_id(idesc, (uint32_t)(kb & 3));
                    const uint64_t a = a_desc + (uint32_t)(stage * (W_BYTES >> 4));
                    const uint64_t b = b_desc + (uint32_t)(stage * (C::X_BYTES >> 4));
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        umma_mxf8<false>(d, a + (a_step >> 4) * k, b + 2u * k, id, sf, sf + 4, kb != kb0 || k != 0 ? 1u : 0u);
                    umma_commit(empty_bar(stage));
                    if (last) umma_commit(sempty_bar(slot));
                }
                __syncwarp();
                if (++stage == stages) stage = 0, phase ^= 1u;
                if (last && ++slot == SF_SLOTS) slot = 0, sphase ^= 1u;
            }
            if (!ok) break;
            if (elect_one()) umma_commit(tfull_bar(acc));
            __syncwarp();
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    } else if (warp == 2) {
        // ------------------------------ scales ------------------------------------
        // one group of four k-blocks ahead, as in rm_fp8_gemm.cu
        const int g0 = kb0 / 4, g1 = (kb1 + 3) / 4;
        struct Words {
            uint32_t x[(NB + 31) / 32], w;
        };
        auto load = [&](int i, int g) {
            const Tile tl = tile_of(i, args);
            const int t = tl.t, nb = tl.n0 / BM;
            Words r;
#pragma unroll
            for (int j = 0; j < (NB + 31) / 32; ++j) {
                const int b = tl.b0 + 32 * j + lane;
                r.x[j] = 0x7f7f7f7fu;
                if (b < args.B)
                    r.x[j] = __ldg(reinterpret_cast<const uint32_t*>(args.xs + ((size_t)b * args.T + t) *
                                                                                  (size_t)args.xs_ld) + g);
            }
            if (TRANS) {
                r.w = __ldg(reinterpret_cast<const uint32_t*>(
                                args.ws + ((size_t)t * args.w_rows + nb) * (size_t)args.ws_ld) + g);
            } else {
                r.w = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int kb = 4 * g + q < args.kblocks ? 4 * g + q : args.kblocks - 1;
                    r.w |= (uint32_t)__ldg(args.ws + ((size_t)t * args.w_rows + kb) * (size_t)args.ws_ld + nb) << (8 * q);
                }
            }
            return r;
        };
        int slot = 0, g = g0, i = unit;
        uint32_t phase = 0;
        Words now{};
        if (i < args.tiles) now = load(i, g0);
        while (i < args.tiles) {
            if (++g == g1) g = g0, i += units;
            Words next{};
            if (i < args.tiles) next = load(i, g);
            if (!wait_bounded(sempty_bar(slot), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) break;
            const uint32_t dst = sSF + slot * SF_BYTES + 16u * lane;
            st_shared_v4(dst, now.w, now.w, now.w, now.w);
            st_shared_v4(dst + 512, now.x[0], NB > 32 ? now.x[(NB > 32)] : 0x7f7f7f7fu,
                         NB > 64 ? now.x[2 * (NB > 64)] : 0x7f7f7f7fu,
                         NB > 64 ? now.x[3 * (NB > 64)] : 0x7f7f7f7fu);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull_bar(slot));
            if (++slot == SF_SLOTS) slot = 0, phase ^= 1u;
            now = next;
        }
    } else {
        // ------------------------------ epilogue ----------------------------------
        constexpr int NS = C::SAMPLES;
        const int quad = warp & 3, tid = 32 * quad + lane, group = (warp - 4) >> 2, j0 = NS * group;
        const uint32_t meet_group = meet_bar + 8u * group;
        int acc = 0;
        uint32_t acc_phase = 0, meet = 0;
        // the four warps of a block wait for one another
        auto all_here = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(meet_group);
            const bool ok = wait_bounded(meet_group, meet, abort_flag, args.err, args.timeout_ns);
            meet ^= 1u;
            return ok;
        };
        for (int i = unit; i < args.tiles; i += units) {
            const Tile tl = tile_of(i, args);
            const int t = tl.t, n0 = tl.n0, n = n0 + tid;
            const float bias = args.bias && n < args.N ? __ldg(args.bias + (size_t)t * args.N + n) : 0.f;
            const int count = args.B - tl.b0 - j0;       // samples of this thread that exist: the first `count` (may be <= 0)
            const size_t row0 = (size_t)(tl.b0 + j0) * args.T + t;
            uint32_t u[EPI == EPI_DGELU ? NS / 2 : 1];   // DGELU: two samples' kept u a word, code and exponent byte each
            if constexpr (EPI == EPI_DGELU) {
                const uint8_t* code = args.o1.codes + row0 * (size_t)args.o1.ld + n;
                const uint8_t* scale = args.o1.scales + row0 * (size_t)args.o1.lds + n0 / kFp8Block;
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    uint32_t w = 127u << 8;
                    if (rank == 0 && j < count && n < args.N) w = __ldg(code) | (uint32_t)__ldg(scale) << 8;
                    u[j / 2] = j % 2 ? u[j / 2] | w << 16 : w;
                    code += (size_t)args.T * (size_t)args.o1.ld;
                    scale += (size_t)args.T * (size_t)args.o1.lds;
                }
            }
            if (!wait_bounded(tfull_bar(acc), acc_phase, abort_flag, args.err, args.timeout_ns)) break;
            tc_fence_after();
            uint32_t r[NS];
            const uint32_t tcol = tmem_base + ((uint32_t)(32 * quad) << 16) + (uint32_t)(acc * NB + j0);
            if constexpr (NS == 16)
                tmem_ld16_nowait(tcol, r);
            else
                tmem_ld32_nowait(tcol, r);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
            if (rank != 0) {                             // the first CTA adds up and finishes
                const uint32_t dst = mapa_shared(sPart + (uint32_t)(rank - 1) * C::PART_BYTES, 0);
                const uint32_t bar = mapa_shared(part_bar, 0);
#pragma unroll
                for (int j = 0; j < NS; j += 4)
                    st_async_v4(dst + 16u * (uint32_t)((j0 + j) / 4 * BM + tid), r[j], r[j + 1], r[j + 2], r[j + 3], bar);
                continue;
            }
            float v[NS];
#pragma unroll
            for (int j = 0; j < NS; ++j) v[j] = __uint_as_float(r[j]);
            if (args.split > 1) {
                if (!wait_bounded(part_bar, 0, abort_flag, args.err, args.timeout_ns)) break;
                mbar_acquire_cluster(part_bar, 0);
                for (int p = 0; p + 1 < args.split; ++p)
#pragma unroll
                    for (int j = 0; j < NS; j += 4) {
                        const uint4 q = ld_shared_u4(sPart + (uint32_t)p * C::PART_BYTES +
                                                     16u * (uint32_t)((j0 + j) / 4 * BM + tid));
                        v[j] += __uint_as_float(q.x);
                        v[j + 1] += __uint_as_float(q.y);
                        v[j + 2] += __uint_as_float(q.z);
                        v[j + 3] += __uint_as_float(q.w);
                    }
            }
            if constexpr (EPI == EPI_DGELU) {
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    const uint32_t w = u[j / 2] >> (16 * (j % 2));
                    v[j] *= fp8_gelu_grad(fp8_unpack2<false>(w & 0xffu).x * fp8_scale(w >> 8 & 0xffu));
                }
            } else {
#pragma unroll
                for (int j = 0; j < NS; ++j) v[j] += bias;
            }
            if constexpr (EPI == EPI_BF16 || EPI == EPI_F32 || EPI == EPI_DGELU) {
                using Out = typename std::conditional<EPI == EPI_F32, float, __nv_bfloat16>::type;
                if (n < args.N) {
                    Out* y = reinterpret_cast<Out*>(args.y) + row0 * (size_t)args.N + n;
                    const size_t step = (size_t)args.T * (size_t)args.N;
#pragma unroll
                    for (int j = 0; j < NS; ++j, y += step) {
                        if (j < count) {
                            if constexpr (EPI == EPI_F32)
                                *y = v[j];
                            else
                                *y = __float2bfloat16_rn(v[j]);
                        }
                    }
                }
            }
            if constexpr (EPI == EPI_GELU || EPI == EPI_GELU_KEEP || EPI == EPI_DGELU) {
                // one 8-bit output: the largest magnitudes of each sample's 128 columns meet,
                // thread j makes sample j's scale, all round by it
                auto save = [&](const Fp8View& out, float (&x)[NS], uint32_t* m) {
                    uint32_t* scale = m + 4 * NB;
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const uint32_t a = __reduce_max_sync(0xffffffffu, fp8_finite_bits(x[j]));
                        if (lane == 0) m[quad * NB + j0 + j] = a;
                    }
                    if (!all_here()) return false;
                    if (tid < NS) {
                        const uint32_t* q = m + j0 + tid;
                        const uint32_t E = fp8_exponent<false>(max(max(q[0], q[NB]), max(q[2 * NB], q[3 * NB])));
                        scale[j0 + tid] = __float_as_uint(fp8_inv_scale(E));
                        if (tid < count)
                            out.scales[(row0 + (size_t)tid * args.T) * (size_t)out.lds + n0 / kFp8Block] = (uint8_t)E;
                    }
                    if (!all_here()) return false;
                    // four samples of four neighbouring columns change places among four lanes, so that
                    // a lane stores four columns of one sample (N is a multiple of 16 here)
                    uint8_t* code = out.codes + (row0 + (size_t)(lane & 3) * args.T) * (size_t)out.ld + (n & ~3);
                    const size_t step = 4 * (size_t)args.T * (size_t)out.ld;
                    const uint32_t pick1 = (lane & 1) ? 0x3715u : 0x6240u, pick2 = (lane & 2) ? 0x3276u : 0x5410u;
#pragma unroll
                    for (int j = 0; j < NS; j += 4, code += step) {
                        const uint4 sc = *reinterpret_cast<const uint4*>(scale + j0 + j);
                        uint32_t c = fp8_pack4<false>(fp8_poison(x[j]) * __uint_as_float(sc.x),
                                                      fp8_poison(x[j + 1]) * __uint_as_float(sc.y),
                                                      fp8_poison(x[j + 2]) * __uint_as_float(sc.z),
                                                      fp8_poison(x[j + 3]) * __uint_as_float(sc.w));
                        c = __byte_perm(c, __shfl_xor_sync(0xffffffffu, c, 1), pick1);
                        c = __byte_perm(c, __shfl_xor_sync(0xffffffffu, c, 2), pick2);
                        if (n < args.N && j + (lane & 3) < count) *reinterpret_cast<uint32_t*>(code) = c;
                    }
                    return true;
                };
                if constexpr (EPI == EPI_GELU_KEEP)
                    if (!save(args.o1, v, red + 5 * NB)) break;
                if constexpr (EPI != EPI_DGELU) {
#pragma unroll
                    for (int j = 0; j < NS; ++j) v[j] = fp8_gelu(v[j]);
                }
                if (!save(args.o0, v, red)) break;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (args.split > 1) cluster_sync_all();      // no CTA leaves while another may still write to its memory
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

template <int EPI, bool TRANS, int NB>
cudaError_t run(const CUtensorMap& mx, const CUtensorMap& mw, Args a, int num_sms, cudaStream_t s) {
    auto k = fp8_stream_kernel<EPI, TRANS, NB>;
    cudaError_t e = smem_attr_once((const void*)k, Cfg<NB>::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const dim3 block(Cfg<NB>::THREADS);
    const int groups = (a.kblocks + 3) / 4;
    a.split = 1, a.groups = groups;
    for (int c = 2; c <= (a.B > 32 ? MAX_SPLIT_64 : MAX_SPLIT) && (long long)c * a.tiles <= num_sms && c <= groups; c *= 2) {
        const int each = (groups + c - 1) / c;
        if ((c - 1) * each < groups &&                         // no CTA is left without k-blocks
            a.tiles <= cluster_occupancy_once((const void*)k, Cfg<NB>::THREADS, Cfg<NB>::SMEM_BYTES, c, num_sms))
            a.split = c, a.groups = each;
    }
    if (a.split == 1) {
        a.stages = Cfg<NB>::STAGES;
        const int ctas = a.tiles < num_sms ? a.tiles : num_sms;
        return launch_k(k, dim3((unsigned)ctas), block, Cfg<NB>::SMEM_BYTES, s, mx, mw, a);
    }
    a.stages = (Cfg<NB>::STAGES * Cfg<NB>::STAGE_BYTES - (a.split - 1) * Cfg<NB>::PART_BYTES) / Cfg<NB>::STAGE_BYTES;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.tiles * a.split));
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = Cfg<NB>::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, mx, mw, a);
}

template <int EPI, bool TRANS>
cudaError_t run_for(const CUtensorMap& mx, const CUtensorMap& mw, const Args& a, int num_sms, cudaStream_t s) {
    // the MMA's N; T = 8, K = 512, N = 2048, one sample: 3.2 us with 16, 3.6 with 32, 4.2 with 64
    if (a.B <= 16) return run<EPI, TRANS, 16>(mx, mw, a, num_sms, s);
    if (EPI == EPI_DGELU || a.B <= 32) return run<EPI, TRANS, 32>(mx, mw, a, num_sms, s);
    if constexpr (EPI != EPI_DGELU) {
        if (a.B <= 64) return run<EPI, TRANS, 64>(mx, mw, a, num_sms, s);
        return run<EPI, TRANS, 128>(mx, mw, a, num_sms, s);
    }
}

}  // namespace f8s

static long long stream_tiles(const Fp8Product& p) {
    const long long m = (p.B + f8s::SAMPLES_MAX - 1) / f8s::SAMPLES_MAX;
    return m * p.T * ((p.N + f8s::BM - 1) / f8s::BM);
}

bool fp8_streams(const Fp8Product& p, const Fp8Device& dev) {
    const long long tiles = stream_tiles(p);
    if (tiles >= (1ll << 30)) return false;
    if (p.epi == FP8_DGELU) return p.B <= kFp8StreamMaxBdU;
    return p.B <= kFp8StreamMaxB || tiles <= dev.num_sms;
}

cudaError_t launch_fp8_stream(const Fp8Product& p, const Fp8Device& dev, cudaStream_t s) {
    using namespace f8s;
    Args a{};
    a.B = p.B, a.T = p.T, a.K = p.K, a.N = p.N;
    a.n_tiles = (p.N + BM - 1) / BM;
    a.kblocks = (p.K + BK - 1) / BK;
    a.m_tiles = (p.B + SAMPLES_MAX - 1) / SAMPLES_MAX;
    a.tiles = (int)stream_tiles(p);
    a.xs = p.x.scales, a.xs_ld = p.x.lds;
    a.ws = p.w.scales, a.ws_ld = p.w.lds;
    const int wr = p.trans ? p.N : p.K, wc = p.trans ? p.K : p.N;
    a.w_rows = (wr + kFp8Block - 1) / kFp8Block;
    a.x_format = p.x.e5m2 ? 1u : 0u;
    a.early = p.follows && pdl_enabled();
    a.bias = p.bias;
    a.y = p.y;
    a.o0 = p.o0, a.o1 = p.o1;
    a.err = dev.err;
    a.timeout_ns = dev.timeout_ns;
    CUtensorMap mx, mw;
    const auto u8t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int rows = p.B <= 16 ? 16 : p.B <= 32 ? 32 : p.B <= 64 ? 64 : 128;
    if (!fp8_tensor_map(&mx, u8t, p.x.codes, p.K, p.B, p.T, p.T * p.x.ld, p.x.ld, BK, rows) ||
        !fp8_tensor_map(&mw, u8t, p.w.codes, wc, wr, p.T, p.w.ld, (long long)wr * p.w.ld, 128, 128))
        return cudaErrorInvalidValue;
    switch (p.epi) {
        case FP8_OUT_BF16:
            return p.trans ? run_for<EPI_BF16, true>(mx, mw, a, dev.num_sms, s)
                           : run_for<EPI_BF16, false>(mx, mw, a, dev.num_sms, s);
        case FP8_OUT_F32:
            return p.trans ? run_for<EPI_F32, true>(mx, mw, a, dev.num_sms, s)
                           : run_for<EPI_F32, false>(mx, mw, a, dev.num_sms, s);
        case FP8_GELU:
            if (p.trans) return cudaErrorNotSupported;
            return p.o1.codes ? run_for<EPI_GELU_KEEP, false>(mx, mw, a, dev.num_sms, s)
                              : run_for<EPI_GELU, false>(mx, mw, a, dev.num_sms, s);
        case FP8_DGELU:
            if (!p.trans) return cudaErrorNotSupported;
            return run_for<EPI_DGELU, true>(mx, mw, a, dev.num_sms, s);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace rm
