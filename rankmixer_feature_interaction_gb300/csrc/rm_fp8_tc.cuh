// tcgen05 forms that the 8-bit kernels add to rm_common.cuh: block-scaled MMA
// on 8-bit operands, the copy of scales into tensor memory, and the shared-
// memory descriptors of 128-byte swizzled operands in both majors.
#pragma once

#include "rm_common.cuh"

namespace rm {

// 3-D tensor map {inner, rows, groups} with boxes of box_inner x box_rows
// elements (128 bytes wide with the 128-byte swizzle, or 64 bytes of codes with
// the 64-byte one); what lies outside reads as zero and is not written.
bool fp8_tensor_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, long long inner, long long rows,
                    long long groups, long long row_bytes, long long group_bytes, int box_inner, int box_rows);

// Operand tile of 128-byte rows written by TMA with the 128-byte swizzle
// (layout type 2, descriptor version 1), base 1024-byte aligned.  K-major: a row
// holds 128 bytes of K of one M (or N) index.  MN-major: a row holds 128 bytes
// of M (or N) of one K index; lbo is the distance between such runs.  In both,
// groups of eight rows lie 1024 bytes apart (stride byte offset).
__device__ __forceinline__ uint64_t sw128_operand(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// 512 bytes of scales (32 rows of 16 bytes, no swizzle): eight-row groups are
// 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    return d;
}

// Instruction descriptor of kind::mxf8f6f4: operand formats (0 e4m3, 1 e5m2) at
// bits 7 and 10, majors (1: MN) at 15 and 16, N >> 3 at 17, exponent-only
// scales at 23, M >> 4 at 24.  with_scale_id selects the byte of the 32-bit
// scale words, at bits 4 (B) and 29 (A).
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, bool a_mn, bool b_mn) {
    return ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t with_scale_id(uint32_t idesc, uint32_t id) { return idesc | (id << 4) | (id << 29); }

template <bool PAIR>
__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
            : "memory");
}

// Scales of 128 rows (one 32-bit word each: row r at 16 (r % 32) + 4 (r / 32))
// into four columns of tensor memory, repeated for the four lane quarters.  As
// a pair, each CTA's tensor memory takes its own shared memory's scales.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// One lane of a converged warp.  Behind this an MMA's issue takes about 25 cycles,
// behind a comparison with the lane's number about 78.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// mbar_wait_bounded that looks at the clock only after some tries: reading the
// global timer takes longer than most of these waits.
// A warp that gives up stays for another millisecond: loads into the CTA's ring, MMAs
// and their commits may still be under way, and must not reach shared or tensor memory
// once these belong to another CTA.  They take microseconds, nothing is issued for long
// after one of the roles has stopped, and the CTA ends only when all of its warps have.
// (At the end of the kernel the same wait cost a register and 3% of the FFN's forward.)
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort, int* err,
                                             uint64_t timeout_ns) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    if (mbar_wait_bounded(bar, parity, abort, err, timeout_ns)) return true;
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
    do {
        __nanosleep(1000);
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    } while (t - t0 < 1000000u);
    return false;
}

// Arrive on the pair's barrier (a shared::cluster address) after writes to this
// CTA's own shared memory that fence_proxy_async_smem has ordered before the
// tensor core's reads of it.  The fence carries the data; the arrival needs no
// cluster-wide release of its own, whose memory barrier costs about 1000 cycles.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One row's 64 bytes into this warp's staging, 16 bytes at a time: piece c of row
// r at c ^ (r / 2 % 4), which keeps rows and pieces free of bank conflicts.
__device__ __forceinline__ uint32_t staged_at(uint32_t stage, int row, int c) {
    return stage + 64u * row + 16u * (uint32_t)(c ^ ((row >> 1) & 3));
}
__device__ __forceinline__ uint4 staged16(uint32_t stage, int row, int c) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(staged_at(stage, row, c)));
    return v;
}

// The staged 32 rows to memory: row r at dst + r pitch, the first `rows` of them,
// of each the first `bytes` (whole 16-byte pieces when VEC, else elements of ESZ
// bytes, neighbouring lanes neighbouring elements).  Plain stores: the staging is
// free again after a warp barrier, where a bulk copy's reads would be waited for.
template <bool VEC, int ESZ>
__device__ __forceinline__ void store_rows(uint32_t stage, char* dst, size_t pitch, int rows, int bytes, int lane) {
    __syncwarp();
    if (VEC) {
        const int c = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            if (r < rows && 16 * c < bytes)
                *reinterpret_cast<uint4*>(dst + (size_t)r * pitch + 16 * c) = staged16(stage, r, c);
        }
    } else {
        constexpr int PER = 64 / ESZ;              // elements of a row's 64 bytes
        const int at = ESZ * (lane % PER);
#pragma unroll 4
        for (int r = lane / PER; r < rows; r += 32 / PER) {
            const uint32_t src = staged_at(stage, r, at >> 4) + (at & 15);
            if (at < bytes) {
                char* p = dst + (size_t)r * pitch + at;
                if (ESZ == 2) {
                    uint16_t v;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src));
                    *reinterpret_cast<uint16_t*>(p) = v;
                } else {
                    uint32_t v;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(src));
                    *reinterpret_cast<uint32_t*>(p) = v;
                }
            }
        }
    }
    __syncwarp();
}

}  // namespace rm
