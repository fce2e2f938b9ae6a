// What the two tensor-core kernels of the 4-bit products share: the block-scaled
// MMA on 4-bit operands, the exponent bytes of a k-block in tensor memory, and the
// tiles of rows that a product walks.
#pragma once

#include <type_traits>

#include "rm_fp4.cuh"
#include "rm_fp8.cuh"
#include "rm_fp8_tc.cuh"

namespace rm {
namespace f4 {

constexpr int BK = kFp4KBlock;           // values of K of a k-block: 128 bytes of codes, four MMAs
constexpr int QUAD_BYTES = 512;          // exponent bytes of 128 rows and 128 values
constexpr int SF_BYTES = 2 * QUAD_BYTES; // ... and of a k-block

// Instruction descriptor of kind::mxf4: both operands e2m1 (format 1 at bits 7 and
// 10), K-major, N >> 3 at 17, exponent-only scales at 23, M >> 4 at 24, K = 64.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

// One step of 64 values of K; the scales are two bytes a row, the lower or the upper
// two (with_scale_id 0 or 2) of its 32-bit words.
template <bool PAIR>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
}

// fp8_gelu of two values, the same bits: the polynomial in x = -|u| = u - 2 relu(u), which
// is exact, so that one variable serves it and the last step.  6.5 instructions a value
// instead of 10 (layer 1 of the FFN at B = 2048 252 us instead of 307; with the sign set
// by a logical instruction a value 262).
__device__ __forceinline__ void fp4_gelu2(float& a, float& b) {
    const uint64_t relu = f2_pack(fmaxf(a, 0.f), fmaxf(b, 0.f)), x = f2_fma(relu, f2_splat(-2.f), f2_pack(a, b));
    uint64_t p = f2_fma(x, f2_splat(9.30538079e-07f), f2_splat(4.20015094e-05f));
    p = f2_fma(x, p, f2_splat(7.80347327e-04f));
    p = f2_fma(x, p, f2_splat(8.01421981e-03f));
    p = f2_fma(x, p, f2_splat(5.32146059e-02f));
    p = f2_fma(x, p, f2_splat(-4.58957642e-01f));
    p = f2_fma(x, p, f2_splat(1.15113652f));
    p = f2_fma(x, p, f2_splat(-9.99999404e-01f));
    float p0, p1;
    f2_unpack(p, p0, p1);
    f2_unpack(f2_fma(x, f2_pack(ex2_approx(p0), ex2_approx(p1)), relu), a, b);
}

// Bytes of blocks that a row does not have become 127 (its codes there are zero, but
// an exponent byte of 255 would make them NaN); left: blocks from this word on.
__device__ __forceinline__ uint32_t existing_blocks(uint32_t w, int left) {
    if (left >= 4) return w;
    if (left <= 0) return 0x7f7f7f7fu;
    const uint32_t keep = (1u << (8 * left)) - 1u;
    return (w & keep) | (0x7f7f7f7fu & ~keep);
}

// Exponent bytes of activations on their way to tensor memory.  Rows may start
// anywhere, so their bytes lie row by row: 16 of them (two k-blocks) a row and step.
// In an operand a row's word of four lies at 16 (r % 32) + 4 (r / 32) of its quad:
// with rows lane, + 32, + 64, + 96 in one lane, its words of a quad are 16 bytes in a
// row, no exchange between lanes.  A lane fetches its rows' bytes DEPTH steps ahead
// (cp.async into a ring of its own) and reads back only what it fetched itself: with
// loads into registers one step ahead the 1B product waited for them, 1.03 ms
// against 0.48.
template <int ROWS, int DEPTH>
struct RowScales {
    static constexpr int STEPS = DEPTH, SLOT = 16 * ROWS, BYTES = DEPTH * SLOT, PER = (ROWS + 31) / 32;
    uint32_t ring, slot = 0;
    uint4 w[PER];
    __device__ __forceinline__ explicit RowScales(uint32_t at) : ring(at) {}
    __device__ __forceinline__ uint32_t mine(int lane) const { return ring + slot * SLOT + 16u * lane; }
    // step g of the first `rows` rows, the first one's bytes at p
    __device__ __forceinline__ void fetch(const uint8_t* p, long long pitch, int rows, int g, int lane) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int m = 32 * j + lane;
            const uint32_t dst = mine(lane) + 512u * j;
            if (m < rows && m < ROWS)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(p + m * pitch + 16ll * g) : "memory");
            else if (m < ROWS)
                st_shared_v4(dst, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
        }
        done();
    }
    // (also where there is nothing left to fetch: take counts on DEPTH groups)
    __device__ __forceinline__ void done() {
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++slot == DEPTH) slot = 0;
    }
    // the oldest of DEPTH fetched steps, which is step g of its rows of nb blocks
    __device__ __forceinline__ void take(int g, int nb, int lane) {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        const int left = nb - 16 * g;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            w[j] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
            if (32 * j + lane < ROWS) w[j] = ld_shared_u4(mine(lane) + 512u * j);
            if (left < 16) {
                w[j].x = existing_blocks(w[j].x, left);
                w[j].y = existing_blocks(w[j].y, left - 4);
                w[j].z = existing_blocks(w[j].z, left - 8);
                w[j].w = existing_blocks(w[j].w, left - 12);
            }
        }
    }
    // half h (k-block 0 or 1 of the two) to shared memory: two quads
    __device__ __forceinline__ void store(uint32_t dst, int h, int lane) const {
        constexpr uint32_t ONE = 0x7f7f7f7fu;
        const uint4 a = w[0], b = PER > 1 ? w[PER > 1] : make_uint4(ONE, ONE, ONE, ONE);
        const uint4 c = PER > 2 ? w[2 * (PER > 2)] : make_uint4(ONE, ONE, ONE, ONE);
        const uint4 d = PER > 3 ? w[3 * (PER > 3)] : make_uint4(ONE, ONE, ONE, ONE);
        if (h == 0) {
            st_shared_v4(dst + 16u * lane, a.x, b.x, c.x, d.x);
            st_shared_v4(dst + QUAD_BYTES + 16u * lane, a.y, b.y, c.y, d.y);
        } else {
            st_shared_v4(dst + 16u * lane, a.z, b.z, c.z, d.z);
            st_shared_v4(dst + QUAD_BYTES + 16u * lane, a.w, b.w, c.w, d.w);
        }
    }
};

}  // namespace f4

// Groups of up to this many rows: the weights are streamed past all of them at once
// (launch_fp4_stream) instead of in tiles of 256 rows by pairs.  In a graph, streamed and
// by pairs: T = 32, K = 1536, N = 6144 27.7 and 39.2 us at 1 sample, 35.0 and 37.4 at 128
// (of 130 samples, two tiles, 48.9 and 37.4); T = 8, K = 512, N = 2048 2.6 and 5.9, 3.5 and
// 6.3; the experts of T = 32, E = 8, D = 1536, F = 2048 131 and 161 us at 8 samples, 180
// and 190 at 128.  Per token with Gelu, whose epilogue grows with the rows, up to 80.  FFNs
// with layer 1 streamed and by pairs: T = 32, D = 1536, F = 6144 77 and 73 us at 80, 81 and 74
// at 96, 91 and 75 at 128; T = 16, D = 512, F = 2048 16.3 and 16.5, 17.2 and 16.6, 18.5 and
// 16.9; T = 4, D = 2048, F = 8192 25.3 and 26.2, 26.2 and 26.2, 27.9 and 26.7.  What has no
// more tiles than SMs stays streamed by the rule below: T = 4, D = 512, F = 2048 12.7 and
// 13.5, 13.2 and 13.6, 13.8 and 13.9.  (Against it: T = 16, D = 512, F = 2432, just two rounds
// of tiles, 17.1 and 19.4, 18.0 and 19.5, 19.3 and 19.7.)
// More samples are streamed too, per token, where that makes no more tiles than two rounds
// of the SMs (one with Gelu): T = 8, K = 512, N = 2048, 256 samples (256 tiles) 4.9 and 6.3
// us, K = 2048, N = 512, 512 samples (128 tiles) 5.3 and 7.2; 512 samples of the first (512
// tiles) 7.8 and 7.3; with Gelu the FFN's 256 tiles took 18.4 us where pairs take 15.0.
constexpr int kFp4StreamMaxB = 128, kFp4StreamMaxGeluB = 80;
bool fp4_streams(const Fp4Product& p, const Fp8Device& dev);
cudaError_t launch_fp4_stream(const Fp4Product& p, const Fp8Device& dev, cudaStream_t s);

}  // namespace rm
