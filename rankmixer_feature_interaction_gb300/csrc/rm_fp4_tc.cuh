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

// Exponent bytes of activations on their way to tensor memory: a lane holds rows
// lane, + 32, + 64, + 96, of each 16 bytes (two k-blocks) as they lie in memory.
// In an operand a row's word lies at 16 (r % 32) + 4 (r / 32) of its quad, so the
// four words of one lane and quad are 16 bytes in a row: no exchange between lanes.
struct RowScales {
    uint4 w[4];
    // half h (k-block 0 or 1 of the two) to shared memory: two quads
    __device__ __forceinline__ void store(uint32_t dst, int h, int lane) const {
        if (h == 0) {
            st_shared_v4(dst + 16u * lane, w[0].x, w[1].x, w[2].x, w[3].x);
            st_shared_v4(dst + QUAD_BYTES + 16u * lane, w[0].y, w[1].y, w[2].y, w[3].y);
        } else {
            st_shared_v4(dst + 16u * lane, w[0].z, w[1].z, w[2].z, w[3].z);
            st_shared_v4(dst + QUAD_BYTES + 16u * lane, w[0].w, w[1].w, w[2].w, w[3].w);
        }
    }
};
// Bytes of blocks that a row does not have become 127 (its codes there are zero, but
// an exponent byte of 255 would make them NaN); left: blocks from this word on.
__device__ __forceinline__ uint32_t existing_blocks(uint32_t w, int left) {
    if (left >= 4) return w;
    if (left <= 0) return 0x7f7f7f7fu;
    const uint32_t keep = (1u << (8 * left)) - 1u;
    return (w & keep) | (0x7f7f7f7fu & ~keep);
}
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, int g, int nb) {
    uint4 v = __ldg(reinterpret_cast<const uint4*>(row) + g);
    const int left = nb - 16 * g;
    if (left < 16) {
        v.x = existing_blocks(v.x, left);
        v.y = existing_blocks(v.y, left - 4);
        v.z = existing_blocks(v.z, left - 8);
        v.w = existing_blocks(v.w, left - 12);
    }
    return v;
}

// A tile of rows of one group: row i lies at (row + i step) of x and of the output,
// its codes at coordinates (row, plane) of x's tensor map.
struct RowTile {
    int g, row, plane, rows;
    long long at;
};

}  // namespace f4

// Groups of up to this many rows: the weights are streamed past all of them at once
// (launch_fp4_stream) instead of in tiles of 256 rows.
constexpr int kFp4StreamMaxB = 128;
cudaError_t launch_fp4_stream(const Fp4Product& p, const Fp8Device& dev, cudaStream_t s);

}  // namespace rm
