// The block quantiser: bf16 or fp32 -> e4m3 codes with a power-of-two scale per
// block of 128, along the rows, along the columns (a transposed result) or
// both from one read.
//
// A CTA takes a 128 x 128 tile of x: thread (g, l), g = 0..15, l = 0..15, holds
// rows 8 g .. 8 g + 7 and columns 8 l .. 8 l + 7.  A block along a row lies in
// the 16 lanes of a half-warp; a block down a column is 8 values in each of 16
// half-warps, whose maxima meet in shared memory.  The transposed codes are
// turned in shared memory, so that both outputs are written in rows of 128
// contiguous bytes.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_format.cuh"
#include "fp8_kernels.h"
#include "ptx.cuh"

namespace wstma {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float half_warp_max(float v)
{
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// One scale byte per row (word [kb/4][row]); the last block's writer fills its word.
__device__ __forceinline__ void store_scale(uint8_t *scales, int64_t rows, int64_t row, int32_t kb, int32_t KB,
                                            uint32_t e)
{
    uint8_t *const word = scales + ((int64_t)(kb >> 2) * rows + row) * 4;
    word[kb & 3] = (uint8_t)e;
    if (kb == KB - 1)
        for (int32_t b = (kb & 3) + 1; b < 4; ++b)
            word[b] = 127;
}

template <bool kFp32, bool kRows, bool kCols>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantizeParams p)
{
    __shared__ float colmax[kCols ? 16 : 1][kFp8Block];
    __shared__ float tilemax[kThreads / 32];
    __shared__ __align__(16) uint8_t turned[kCols ? kFp8Block * kFp8Block : 16];
    grid_dependency_wait();
    grid_launch_dependents();
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
    const uint32_t col_tiles = (uint32_t)(p.C + kFp8Block - 1) / kFp8Block;
    const int32_t rb = (int32_t)(blockIdx.x / col_tiles), cb = (int32_t)(blockIdx.x % col_tiles);
    const int32_t r0 = rb * kFp8Block + g * 8, c0 = cb * kFp8Block + l * 8;
    const int32_t R = p.R, C = p.C;

    float y[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i;
        if (r < R && c0 < C) {
            if constexpr (kFp32)
                load8_float(static_cast<const float *>(p.x) + r * p.ldx, c0, C, p.x_vec, y[i]);
            else
                unpack8(load8_bf16(static_cast<const uint16_t *>(p.x) + r * p.ldx, c0, C, p.x_vec), y[i]);
            if (p.row_factor) {
                const float f = p.row_factor[r];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[i][j] *= f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[i][j] = 0.f;
        }
    }
    if (p.column_factor && c0 < C) {
        float f[8];
        if (p.column_fp32)
            load8_float(static_cast<const float *>(p.column_factor), c0, C, false, f);
        else
            unpack8(load8_bf16(static_cast<const uint16_t *>(p.column_factor), c0, C, false), f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[i][j] *= c0 + j < C ? f[j] : 0.f;
    }

    // Infinities are rare: one vote for the CTA decides whether they become NaN
    // here, so that the maxima below are over finite values.
    bool inf = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            inf = inf || is_inf(y[i][j]);
    if (inf) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[i][j] = inf_to_nan(y[i][j]);
    }

    float rmax[8], cmax[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        cmax[j] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        rmax[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rmax[i] = fmaxf(rmax[i], fabsf(y[i][j]));
            cmax[j] = fmaxf(cmax[j], fabsf(y[i][j]));
        }
    }

    if (p.tile) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, rmax[i]);
        m = half_warp_max(m);
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        if ((threadIdx.x & 31) == 0)
            tilemax[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k)
            m = fmaxf(m, tilemax[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            rmax[i] = cmax[i] = m;
    } else {
        if constexpr (kRows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                rmax[i] = half_warp_max(rmax[i]);
        }
        if constexpr (kCols) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                colmax[g][l * 8 + j] = cmax[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    cmax[j] = fmaxf(cmax[j], colmax[k][l * 8 + j]);
        }
    }

    if constexpr (kRows) {
        const int32_t KB = (C + kFp8Block - 1) / kFp8Block;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + i;
            if (r >= R)
                break;
            const uint32_t e = scale_byte(rmax[i]);
            const float up = scale_inverse(e);
            if (c0 < C)
                store8_codes(p.codes + r * p.ldq, c0, C,
                             make_uint2(pack_e4m3x4(y[i][0] * up, y[i][1] * up, y[i][2] * up, y[i][3] * up),
                                        pack_e4m3x4(y[i][4] * up, y[i][5] * up, y[i][6] * up, y[i][7] * up)));
            if (l == 0)
                store_scale(p.scales, R, r, cb, KB, e);
        }
    }
    if constexpr (kCols) {
        // row c of the turned tile: 16 units of 8 bytes, unit u at u ^ (c / 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t e = scale_byte(cmax[j]);
            const float up = scale_inverse(e);
            const uint2 q = make_uint2(pack_e4m3x4(y[0][j] * up, y[1][j] * up, y[2][j] * up, y[3][j] * up),
                                       pack_e4m3x4(y[4][j] * up, y[5][j] * up, y[6][j] * up, y[7][j] * up));
            *reinterpret_cast<uint2 *>(turned + (l * 8 + j) * kFp8Block + ((g ^ l) << 3)) = q;
            if (g == 0 && c0 + j < C)
                store_scale(p.scales_t, C, c0 + j, rb, (R + kFp8Block - 1) / kFp8Block, e);
        }
        __syncthreads();
        // half-warp g writes rows 8 g .. 8 g + 7 of the turned tile, 8 bytes a lane
        const int32_t rl = rb * kFp8Block + l * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = (int64_t)cb * kFp8Block + g * 8 + i;
            if (c < C && rl < R)
                store8_codes(p.codes_t + c * p.ldqt, rl, R,
                             *reinterpret_cast<const uint2 *>(turned + (g * 8 + i) * kFp8Block + ((l ^ g) << 3)));
        }
    }
}

}  // namespace

int launch_quantize(const QuantizeParams &p, cudaStream_t stream)
{
    const bool rows = p.codes != nullptr, cols = p.codes_t != nullptr;
    void (*fn)(QuantizeParams) = nullptr;
    if (p.x_fp32)
        fn = rows ? (cols ? &quantize_kernel<true, true, true> : &quantize_kernel<true, true, false>)
                  : &quantize_kernel<true, false, true>;
    else
        fn = rows ? (cols ? &quantize_kernel<false, true, true> : &quantize_kernel<false, true, false>)
                  : &quantize_kernel<false, false, true>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int64_t tiles = (((int64_t)p.C + kFp8Block - 1) / kFp8Block) * (((int64_t)p.R + kFp8Block - 1) / kFp8Block);
    if (tiles > 0x7FFFFFFFLL)
        return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)tiles, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace wstma
