// What the kernels for few tokens share (ffn_stream.cu, ffn_stream_back.cu): loads of weights that are
// read once and of tokens that every warp reads, and the MMA on registers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace wstma {

// Not through the read-only path: what the kernel before wrote may have been read there.
__device__ __forceinline__ uint4 load_once(const uint16_t *p)
{
    uint4 q;
    asm volatile("ld.global.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "l"(p));
    return q;
}

__device__ __forceinline__ uint4 load_again_16(const uint16_t *p)
{
    uint4 q;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                 : "l"(p));
    return q;
}

__device__ __forceinline__ uint2 load_again_8(const uint16_t *p)
{
    uint2 q;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
    return q;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace wstma
