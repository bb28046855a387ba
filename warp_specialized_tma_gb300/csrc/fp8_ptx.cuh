// Inline PTX of the block-scaled product beside ptx.cuh: the tcgen05.mma kind
// with a scale per block, and the copy of scales from shared to tensor memory.
#pragma once

#include "ptx.cuh"

namespace wstma {

// Watchdog role code of the warp that brings the scales (see WaitCtl).
constexpr uint32_t kRoleScales = 9;

// D[tmem] (+)= (A * sA) (B * sB)^T over 32 elements of k: e4m3 operands in
// shared memory, one e8m0 scale per row for these 32 in tensor memory, fp32 sums.
template <int CG>
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                "r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
            : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (bits 7..9 and 10..12
// = 0), both K-major (bits 15, 16 = 0), N >> 3 in bits 17..22, e8m0 scales (bit
// 23 = 1), M >> 4 in bits 24..28; the byte of the scale words that applies goes
// into bits 4..5 (B) and 29..30 (A), see scale_id().
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N)
{
    return ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

__host__ __device__ constexpr uint32_t scale_id(uint32_t byte) { return (byte << 4) | (byte << 29); }

// 32 rows of 16 contiguous bytes of shared memory -> 4 columns of tensor memory,
// the same in all four lane quadrants: row r's word j lands in lane r, column j.
// In paired mode each CTA of the pair copies from its own shared memory.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Shared-memory descriptor of such a 512-byte block: no swizzle, groups of 8
// rows 128 bytes apart (bits 32..45), descriptor version 1 (46..48).
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1u << 46);
}

// Wait until at most one committed bulk store of this thread still reads shared memory.
__device__ __forceinline__ void bulk_wait_read_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

}  // namespace wstma
