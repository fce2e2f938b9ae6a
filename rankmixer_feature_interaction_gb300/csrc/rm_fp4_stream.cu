// Products of 4-bit operands for few rows a group: the product of rm_fp4_gemm.cu with
// W's rows (the columns of Y) as the rows of the MMA, so that a group's weights are
// streamed once and little is computed for rows that are not there.
//   acc[n][i] = sum_k W[g][n][k] x[row i][k],  128 columns n x NB rows a tile
// Bound by memory: W is read once (0.53 bytes a weight), so the kernel is a deep
// pipeline of weight tiles: one persistent CTA per SM, per k-block of 256 values and
// stage 16 KB of W's codes, 1 KB of its exponent bytes and NB rows of x.
//   warp 0       TMA producer of W: codes, and exponent bytes as they lie
//   warp 1       MMA issuer (tcgen05.mma kind::mxf4, M = 128, N = NB, one CTA)
//   warp 2       x's exponent bytes (RowScales)
//   warp 3       TMA producer of x's codes
//   warps 4-7 (to 11 for more than 16 rows, to 19 for more than 64)  epilogue: a
//                thread owns one column n of 16 or 32 rows; a block of 32 columns of a
//                4-bit output is a warp, which finds its largest value by one warp
//                maximum and turns eight rows' codes in three exchanges
// The kernel is launched while its predecessor may still run.  Where that predecessor
// is one of this library's own launches of the same call, W was in memory before it
// began, and the experts' tiles too (the sort is the launch before it or an earlier one,
// and it waited for that one's end before this kernel could start): warp 0 starts on W at
// once, everything else waits for the predecessor's end.
// Measured (in a graph, bf16 out): T = 32, K = 1536, N = 6144 27.7 us at 1 sample (160 MB:
// 5.8 TB/s), 31.9 at 64, 35.0 at 128; K = 6144, N = 1536 (384 tiles, 2.5 rounds of the SMs)
// 29.1, 30.1, 32.5; the experts of T = 32, E = 8, K = 1536, N = 2048 at 8 samples 54 us for
// 384 MB of open weights, 7.1 TB/s.  The rest at one sample is the last, partly filled
// round (11 where 10.1 would do) and the start.  Dividing that round's tiles into quarters
// of 32 columns made it slower (29 to 39 us): a k-block's chain of loads, exponent bytes
// and MMAs takes as long for a quarter.
// Every mbarrier wait is bounded in time; on expiry the CTA latches an error
// word and all roles unwind.
#include <cudaTypedefs.h>

#include "rm_fp4_tc.cuh"

namespace rm {
namespace f4s {
using namespace f4;

constexpr int BM = 128;                      // columns of Y per tile
constexpr int W_BYTES = BM * 128;

template <int NB>
struct Cfg {
    static constexpr int X_BYTES = NB * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES + 2 * SF_BYTES;
    using Scales = RowScales<NB, 8>;
    static constexpr int FIT = (225 * 1024 - Scales::BYTES) / STAGE_BYTES;
    static constexpr int STAGES = FIT < 12 ? FIT : 12;
    static constexpr int EPI_WARPS = NB == 16 ? 4 : NB == 128 ? 16 : 8;
    static constexpr int TMEM_COLS = NB == 128 ? 512 : 256, SF_COL = 2 * NB;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int ROWS = NB / (EPI_WARPS / 4);               // per epilogue thread
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + Scales::BYTES + 512;
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
    static_assert(SF_COL + 32 <= TMEM_COLS, "two accumulators and two slots of exponent bytes");
};

struct Args {
    int B, G, N;
    int n_tiles, m_tiles, kblocks, nb;
    uint32_t tiles;                      // per token
    const int4* table;                   // experts: as in rm_fp4_gemm.cu
    long long n, step;
    const uint8_t* xs;
    long long xs_ld;
    const uint8_t* ws;                   // W's: k-block kb of tile i of group g at ((g n_tiles + i) quads + 2 kb) 512
    long long quads;
    bool early;                          // W may be read before the predecessor's end
    const float* bias;
    void* y;
    Fp4View o;
    int* err;
    unsigned long long timeout_ns;
};

struct Tile {
    int g, m0, rows, n0;
};
// Tiles of rows fastest (per token): those that share a weight tile run side by side.
template <bool EXPERTS>
__device__ __forceinline__ Tile tile_of(uint32_t i, const Args& a) {
    Tile t;
    t.m0 = 0;
    if (!EXPERTS && a.m_tiles > 1) {
        const uint32_t q = i / (uint32_t)a.m_tiles;
        t.m0 = (int)(i - q * a.m_tiles) * kFp4StreamMaxB;
        i = q;
    }
    const uint32_t l = i / (uint32_t)a.n_tiles;
    t.n0 = (int)(i - l * a.n_tiles) * BM;
    if (EXPERTS) {
        const int4 e = __ldg(a.table + 1 + l);
        t.g = e.x, t.m0 = e.y;
        t.rows = (int)min((long long)e.z, a.n - e.y);
    } else {
        t.g = (int)l;
        t.rows = a.B - t.m0;
    }
    return t;
}
template <bool EXPERTS>
__device__ __forceinline__ long long row_of(const Tile& t, int i, const Args& a) {
    return EXPERTS ? (long long)t.m0 + i : (long long)(t.m0 + i) * a.G + t.g;
}

// Eight rows' codes of one column each in a lane to eight columns' of one row: lane
// 8 q + i ends with row i, columns 8 q on.
__device__ __forceinline__ uint32_t turn8(uint32_t w, int lane) {
    uint32_t p = __shfl_xor_sync(0xffffffffu, w, 1);
    w = lane & 1 ? (w & 0xf0f0f0f0u) | ((p >> 4) & 0x0f0f0f0fu) : (w & 0x0f0f0f0fu) | ((p << 4) & 0xf0f0f0f0u);
    p = __shfl_xor_sync(0xffffffffu, w, 2);
    w = __byte_perm(w, p, lane & 2 ? 0x3715u : 0x6240u);
    p = __shfl_xor_sync(0xffffffffu, w, 4);
    return __byte_perm(w, p, lane & 4 ? 0x3276u : 0x5410u);
}

template <int EPI, int NB, bool EXPERTS>
__global__ void __launch_bounds__(Cfg<NB>::THREADS, 1)
fp4_stream_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Args args) {
    using C = Cfg<NB>;
    constexpr int STAGES = C::STAGES, EPI_WARPS = C::EPI_WARPS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* base_ptr = smem_raw + (base - raw_addr);
    const uint32_t sW = base, sX = sW + STAGES * W_BYTES, sSFW = sX + STAGES * C::X_BYTES, sSFX = sSFW + STAGES * SF_BYTES;
    const uint32_t sRing = sSFX + STAGES * SF_BYTES, bar0 = sRing + C::Scales::BYTES;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + x); };
    auto tempty_bar = [&](int x) { return bar0 + 8u * (2 * STAGES + 2 + x); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(base_ptr + (bar0 + 8u * (2 * STAGES + 4) - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 3);            // W's bytes, x's bytes, x's exponent bytes
            mbar_init(empty_bar(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(tfull_bar(x), 1);
            mbar_init(tempty_bar(x), EPI_WARPS);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
    const int kblocks = args.kblocks;
    const uint32_t units = gridDim.x;
    if (!(args.early && warp == 0)) {
        pdl_wait();
        pdl_launch_next();
    }
    const uint32_t tiles = EXPERTS ? (uint32_t)__ldg(&args.table[0].x) * (uint32_t)args.n_tiles : args.tiles;

    if (warp == 0 || warp == 3) {
        // ------------------------------ TMA producers -----------------------------
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        Tile next{};
        if (blockIdx.x < tiles) next = tile_of<EXPERTS>(blockIdx.x, args);
        for (uint32_t i = blockIdx.x; ok && i < tiles; i += units) {
            const Tile tl = next;
            if (i + units < tiles) next = tile_of<EXPERTS>(i + units, args);
            const uint8_t* sf = args.ws + (((long long)tl.g * args.n_tiles + tl.n0 / BM) * args.quads) * QUAD_BYTES;
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (warp == 0) {
                        mbar_arrive_expect_tx(full_bar(stage), W_BYTES + SF_BYTES);
                        tma_load_3d(&tmW, sW + stage * W_BYTES, full_bar(stage), kb * 128, tl.n0, tl.g);
                        bulk_copy_g2s(sSFW + stage * SF_BYTES, sf + (size_t)kb * SF_BYTES, SF_BYTES, full_bar(stage));
                    } else {
                        mbar_arrive_expect_tx(full_bar(stage), C::X_BYTES);
                        tma_load_3d(&tmX, sX + stage * C::X_BYTES, full_bar(stage), kb * 128, tl.m0, EXPERTS ? 0 : tl.g);
                    }
                }
                __syncwarp();
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer --------------------------------
        const uint32_t idesc = idesc_mxf4(BM, NB);
        const uint64_t a_desc = sw128_operand(sW, 16u), b_desc = sw128_operand(sX, 16u);
        const uint64_t sfa_desc = scale_desc(sSFW), sfb_desc = scale_desc(sSFX);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0, slot = 0;
        bool ok = true;
        for (uint32_t i = blockIdx.x; ok && i < tiles; i += units) {
            if (!wait_bounded(tempty_bar(acc), acc_phase ^ 1u, abort_flag, args.err, args.timeout_ns)) break;
            tc_fence_after();
            const uint32_t d = tmem_base + (uint32_t)(acc * NB);
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!wait_bounded(full_bar(stage), phase, abort_flag, args.err, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sf = tmem_base + C::SF_COL + 16u * slot;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t at = (uint32_t)((stage * SF_BYTES + q * QUAD_BYTES) >> 4);
                        copy_scales<false>(sf + 4u * q, sfa_desc + at);
                        copy_scales<false>(sf + 8u + 4u * q, sfb_desc + at);
                    }
                    const uint64_t a = a_desc + (uint32_t)(stage * (W_BYTES >> 4));
                    const uint64_t b = b_desc + (uint32_t)(stage * (C::X_BYTES >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_mxf4<false>(d, a + 2u * k, b + 2u * k, with_scale_id(idesc, 2u * (k & 1)), sf + 4u * (k >> 1),
                                         sf + 8u + 4u * (k >> 1), (kb | k) != 0 ? 1u : 0u);
                    umma_commit(empty_bar(stage));
                }
                __syncwarp();
                slot ^= 1u;
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
            if (!ok) break;
            if (elect_one()) umma_commit(tfull_bar(acc));
            __syncwarp();
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    } else if (warp == 2) {
        // ------------------------------ scales of x -------------------------------
        const int groups = (kblocks + 1) / 2;
        typename C::Scales sc(sRing);
        uint32_t i = blockIdx.x;                         // of the next step to fetch
        int g = 0;
        Tile tl{};
        if (i < tiles) tl = tile_of<EXPERTS>(i, args);
        auto fetch = [&]() {
            if (i >= tiles) return sc.done();
            sc.fetch(args.xs + row_of<EXPERTS>(tl, 0, args) * args.xs_ld, args.step * args.xs_ld, tl.rows, g, lane);
            if (++g == groups) {
                g = 0, i += units;
                if (i < tiles) tl = tile_of<EXPERTS>(i, args);
            }
        };
#pragma unroll 1
        for (int d = 0; d < C::Scales::STEPS; ++d) fetch();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (uint32_t j = blockIdx.x; ok && j < tiles; j += units)
            for (int kb = 0; ok && kb < kblocks; kb += 2) {
                sc.take(kb / 2, args.nb, lane);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (kb + h >= kblocks) break;
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, args.err, args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    sc.store(sSFX + stage * SF_BYTES, h, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full_bar(stage));
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
                fetch();
            }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------ epilogue ----------------------------------
        constexpr int NS = C::ROWS;
        const int quad = warp & 3, j0 = NS * ((warp - 4) >> 2);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (uint32_t i = blockIdx.x; i < tiles; i += units) {
            const Tile tl = tile_of<EXPERTS>(i, args);
            const int n = tl.n0 + 32 * quad + lane;
            const float bias = args.bias && n < args.N ? __ldg(args.bias + (size_t)tl.g * args.N + n) : 0.f;
            const int count = tl.rows - j0;            // rows of this thread that exist: the first `count` (may be <= 0)
            const long long row0 = row_of<EXPERTS>(tl, j0, args);
            if (!wait_bounded(tfull_bar(acc), acc_phase, abort_flag, args.err, args.timeout_ns)) break;
            tc_fence_after();
            uint32_t r[NS];
            const uint32_t tcol = tmem_base + ((uint32_t)(32 * quad) << 16) + (uint32_t)(acc * NB + j0);
            if constexpr (NS == 16) {
                tmem_ld16_nowait(tcol, r);
                tmem_wait_ld16(r);
            } else {
                tmem_ld32_nowait(tcol, r);
                tmem_wait_ld32(r);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
            if (count <= 0) continue;
            if constexpr (EPI == FP4_GELU) {
                // N is a multiple of 32: a warp's columns exist or do not
                if (n - lane >= args.N) continue;
                uint32_t mine = 127;
#pragma unroll
                for (int j = 0; j < NS; j += 8) {
                    if (j >= count) break;
                    float q[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) q[k] = __uint_as_float(r[j + k]) + bias;
#pragma unroll
                    for (int k = 0; k < 8; k += 2) fp4_gelu2(q[k], q[k + 1]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t E = fp4_exponent(__reduce_max_sync(0xffffffffu, fp4_abs_bits(q[k])));
                        if (lane == j + k) mine = E;
                        q[k] *= fp4_inv_scale(E);
                    }
                    const uint32_t w = turn8(fp4_pack8(q), lane);
                    if (j + (lane & 7) < count)
                        *reinterpret_cast<uint32_t*>(args.o.codes + (row0 + (j + (lane & 7)) * args.step) * args.o.ld +
                                                     (n - lane) / 2 + 4 * (lane >> 3)) = w;
                }
                if (lane < NS && lane < count)
                    args.o.scales[(row0 + lane * args.step) * args.o.lds + n / kFp4Block] = (uint8_t)mine;
            } else {
                using Out = typename std::conditional<EPI == FP4_OUT_F32, float, __nv_bfloat16>::type;
                if (n < args.N) {
                    Out* y = static_cast<Out*>(args.y) + row0 * args.N + n;
                    const long long step = args.step * args.N;
#pragma unroll
                    for (int j = 0; j < NS; ++j, y += step)
                        if (j < count) *y = from_f32<Out>(__uint_as_float(r[j]) + bias);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

template <int EPI, int NB, bool EXPERTS>
cudaError_t run(const CUtensorMap& mx, const CUtensorMap& mw, const Args& a, int num_sms, cudaStream_t s) {
    auto k = fp4_stream_kernel<EPI, NB, EXPERTS>;
    const cudaError_t e = smem_attr_once((const void*)k, Cfg<NB>::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const uint32_t ctas = EXPERTS || a.tiles > (uint32_t)num_sms ? (uint32_t)num_sms : a.tiles;
    return launch_k(k, dim3(ctas), dim3(Cfg<NB>::THREADS), Cfg<NB>::SMEM_BYTES, s, mx, mw, a);
}

template <int EPI, bool EXPERTS>
cudaError_t run_for(const CUtensorMap& mx, const CUtensorMap& mw, const Args& a, int num_sms, cudaStream_t s) {
    if (a.B <= 16) return run<EPI, 16, EXPERTS>(mx, mw, a, num_sms, s);
    if (a.B <= 32) return run<EPI, 32, EXPERTS>(mx, mw, a, num_sms, s);
    if (a.B <= 64) return run<EPI, 64, EXPERTS>(mx, mw, a, num_sms, s);
    return run<EPI, 128, EXPERTS>(mx, mw, a, num_sms, s);
}

}  // namespace f4s

bool fp4_streams(const Fp4Product& p, const Fp8Device& dev) {
    if (p.B <= (p.epi == FP4_GELU && !p.tiles ? kFp4StreamMaxGeluB : kFp4StreamMaxB)) return true;
    const long long m = (p.B + kFp4StreamMaxB - 1) / kFp4StreamMaxB, n = (p.N + f4s::BM - 1) / f4s::BM;
    return !p.tiles && m * n * p.G <= (p.epi == FP4_GELU ? 1 : 2) * dev.num_sms;
}

cudaError_t launch_fp4_stream(const Fp4Product& p, const Fp8Device& dev, cudaStream_t s) {
    using namespace f4s;
    Args a{};
    a.B = p.B, a.G = p.G, a.N = p.N;
    a.n_tiles = (p.N + BM - 1) / BM;
    a.kblocks = (p.K + BK - 1) / BK;
    a.nb = (int)fp4_blocks(p.K);
    a.m_tiles = p.tiles ? 1 : (p.B + kFp4StreamMaxB - 1) / kFp4StreamMaxB;
    const long long tiles = (long long)p.G * a.n_tiles * a.m_tiles;
    if (tiles >= 1ll << 31) return cudaErrorNotSupported;        // more tiles than a device's memory holds weights for
    a.tiles = (uint32_t)tiles;
    a.table = p.tiles;
    a.n = p.n;
    a.step = p.tiles ? 1 : p.G;
    a.xs = p.x.scales, a.xs_ld = p.x.lds;
    a.ws = p.w.scales, a.quads = p.w.lds;
    a.early = p.follows && pdl_enabled();
    a.bias = p.bias;
    a.y = p.y;
    a.o = p.o;
    a.err = dev.err;
    a.timeout_ns = dev.timeout_ns;
    const auto u8t = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const long long wide = 16ll * a.nb;
    const int rows = p.B <= 16 ? 16 : p.B <= 32 ? 32 : p.B <= 64 ? 64 : 128;
    CUtensorMap mx, mw;
    const bool ok = (p.tiles ? fp8_tensor_map(&mx, u8t, p.x.codes, wide, p.n, 1, p.x.ld, p.x.ld, 128, rows)
                             : fp8_tensor_map(&mx, u8t, p.x.codes, wide, p.B, p.G, p.G * p.x.ld, p.x.ld, 128, rows)) &&
                    fp8_tensor_map(&mw, u8t, p.w.codes, wide, p.N, p.G, p.w.ld, p.N * p.w.ld, 128, BM);
    if (!ok) return cudaErrorInvalidValue;
    switch (p.epi) {
        case FP4_OUT_BF16:
            return p.tiles ? run_for<FP4_OUT_BF16, true>(mx, mw, a, dev.num_sms, s)
                           : run_for<FP4_OUT_BF16, false>(mx, mw, a, dev.num_sms, s);
        case FP4_OUT_F32:
            return p.tiles ? run_for<FP4_OUT_F32, true>(mx, mw, a, dev.num_sms, s)
                           : run_for<FP4_OUT_F32, false>(mx, mw, a, dev.num_sms, s);
        case FP4_GELU:
            return p.tiles ? run_for<FP4_GELU, true>(mx, mw, a, dev.num_sms, s)
                           : run_for<FP4_GELU, false>(mx, mw, a, dev.num_sms, s);
    }
    return cudaErrorNotSupported;
}

}  // namespace rm
