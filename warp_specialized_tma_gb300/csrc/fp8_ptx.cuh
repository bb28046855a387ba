// Inline PTX of the block-scaled product beside ptx.cuh: the tcgen05.mma kind
// with a scale per block, and the copy of scales from shared to tensor memory.
#pragma once

#include "ptx.cuh"

namespace wstma {

// Watchdog role code of the warp that brings the scales (see WaitCtl).
constexpr uint32_t kRoleScales = 9;

// The MMA issuer runs as a whole, converged warp, and these act for one elected
// lane by a predicate instead of a branch: so the compiler keeps descriptors and
// addresses in uniform registers, where the tensor core reads them.  From a
// branch that one lane takes, every operand of every MMA is first moved there:
// 70 clocks an MMA and 190 a commit, measured on GB300, which bounded the kernel.

// 1 in one lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

// D[tmem] (+)= (A * sA) (B * sB)^T over a block of 128 elements of k, as four MMAs of 32:
// e4m3 operands in shared memory (32 bytes of a swizzled row apart), one e8m0 scale
// per row in tensor memory, fp32 sums.  The first adds to D if `accumulate`.  Probes
// the barrier of the next block on the way, so that the probe's 95 clocks pass
// while the MMAs issue: 1 if its phase has completed.
template <int CG>
__device__ __forceinline__ uint32_t mma_mxf8_block(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                   uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate,
                                                   uint32_t leader, uint32_t next_bar, uint32_t next_parity)
{
    uint32_t ready;
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q, w;\n\t.reg .u64 a, b;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 w, [%9], %10;\n\t"
            "setp.ne.b32 p, %7, 0;\n\t"
            "setp.ne.b32 q, %8, 0;\n\t"
            "mov.u64 a, %2;\n\tmov.u64 b, %3;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
            "setp.ne.b32 p, 1, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "selp.u32 %0, 1, 0, w;\n\t}"
            : "=r"(ready)
            : "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate), "r"(leader),
              "r"(next_bar), "r"(next_parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q, w;\n\t.reg .u64 a, b;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 w, [%9], %10;\n\t"
            "setp.ne.b32 p, %7, 0;\n\t"
            "setp.ne.b32 q, %8, 0;\n\t"
            "mov.u64 a, %2;\n\tmov.u64 b, %3;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
            "setp.ne.b32 p, 1, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "add.u64 a, a, 2;\n\tadd.u64 b, b, 2;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%1], a, b, %4, [%5], [%6], p;\n\t"
            "selp.u32 %0, 1, 0, w;\n\t}"
            : "=r"(ready)
            : "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate), "r"(leader),
              "r"(next_bar), "r"(next_parity)
            : "memory");
    return ready;
}

// mma_commit (CG = 1) or mma_commit_pair (CG = 2) of the elected lane.
template <int CG>
__device__ __forceinline__ void mma_commit_elected(uint32_t bar, uint32_t leader)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
            "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
                bar),
            "h"((uint16_t)0x3), "r"(leader)
            : "memory");
}

// mbar_arrive_expect_tx and the 2-D TMA load of the elected lane; in paired mode the
// bytes complete on a barrier of either CTA, given by its shared::cluster address.
__device__ __forceinline__ void expect_tx_elected(uint32_t bar, uint32_t bytes, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(leader)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tma_load_2d_elected(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y,
                                                    uint32_t bar, uint32_t leader)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(leader)
            : "memory");
}

// Waits, up to `tries` probes of `suspend_ns` each, for the phase with this
// parity; 0 if it did not complete.  A loop inside one statement: the warp
// stays converged around it.
__device__ __forceinline__ uint32_t mbar_wait_tries(uint32_t bar, uint32_t parity, uint32_t suspend_ns, uint32_t tries)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %4;\n\t"
        "WAIT:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra WAIT;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(suspend_ns), "r"(tries)
        : "memory");
    return ok;
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
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc, uint32_t leader)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
            "l"(desc), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
            "l"(desc), "r"(leader)
            : "memory");
}

// Shared-memory descriptor of such a 512-byte block: no swizzle, groups of 8
// rows 128 bytes apart (bits 32..45), descriptor version 1 (46..48).
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1u << 46);
}

// Contiguous copy of `bytes` (a multiple of 16; both addresses 16-byte aligned)
// from global to this CTA's shared memory, completing them on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

}  // namespace wstma
