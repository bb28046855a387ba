// Residual addition, root-mean-square norm and 8-bit quantisation in one pass,
// and the norm's gradients.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_format.cuh"
#include "fp8_kernels.h"
#include "ptx.cuh"

namespace wstma {

namespace {

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Sum over the threads of a row: the warp's when the row is a warp's, else the CTA's.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = warp_sum(v);
    if constexpr (kWarpRow) {
        return v;
    } else {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = (int)blockDim.x >> 5;
        __syncthreads();  // the previous row's sums have been read
        if (lane == 0)
            red[warp] = v;
        __syncthreads();
        return warp_sum(lane < n ? red[lane] : 0.f);
    }
}

__device__ __forceinline__ void load8_weight(const void *w, int fp32, int32_t c, int32_t C, bool vec, float (&f)[8])
{
    if (fp32)
        load8_float(static_cast<const float *>(w), c, C, vec, f);
    else
        unpack8(load8_bf16(static_cast<const uint16_t *>(w), c, C, vec), f);
}

// Vector v of a row (8 columns each): thread t of the row's T holds vectors t,
// t + T, ..., so the 16 lanes of a half-warp always hold one block of 128.
template <int V, bool kWarpRow, bool kRes>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormParams p)
{
    __shared__ float red[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int T = kWarpRow ? 32 : (int)blockDim.x;
    const int t = kWarpRow ? (int)(threadIdx.x & 31u) : (int)threadIdx.x;
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.R)
        return;  // whole warps, and only where rows are warps
    const bool vec = p.vec != 0;
    const int32_t C = p.C;
    const uint16_t *const xr = p.x + row * p.ldx;
    const uint16_t *const rr = kRes ? p.residual + row * p.ldr : nullptr;

    uint4 hv[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        hv[i] = load8_bf16(xr, (t + i * T) * 8, C, vec);
    if constexpr (kRes) {
        uint4 rv[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            rv[i] = load8_bf16(rr, (t + i * T) * 8, C, vec);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float a[8], b[8];
            unpack8(hv[i], a);
            unpack8(rv[i], b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                a[j] += b[j];
            hv[i] = make_uint4(bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(a[4], a[5]),
                               bf16_pair(a[6], a[7]));
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float a[8];
        unpack8(hv[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sum = fmaf(a[j], a[j], sum);
        if constexpr (kRes)
            if ((t + i * T) * 8 < C)
                store8_bf16(p.h + row * p.ldh, (t + i * T) * 8, C, vec, hv[i]);
    }
    sum = row_sum<kWarpRow>(sum, red);
    const float rstd = 1.f / sqrtf(sum / (float)C + p.eps);
    if (p.rstd && t == 0)
        p.rstd[row] = rstd;

    const int32_t KB = (C + kFp8Block - 1) / kFp8Block;
    uint8_t *const codes = p.codes + row * p.ldq;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t c = (t + i * T) * 8;
        float y[8], w[8];
        unpack8(hv[i], y);
        load8_weight(p.weight, p.w_fp32, c, C, vec, w);
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = y[j] * rstd * w[j];
            amax = fmaxf(amax, fabsf(y[j]));
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        if (__any_sync(0xFFFFFFFFu, is_inf(amax))) {
            // a block with an infinity: its scale is that of its finite values
            amax = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                amax = fmaxf(amax, finite_abs(y[j]));
                y[j] = inf_to_nan(y[j]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        }
        const uint32_t e = scale_byte(amax);
        const float up = scale_inverse(e);
        if (c < C) {
            store8_codes(codes, c, C,
                         make_uint2(pack_e4m3x4(y[0] * up, y[1] * up, y[2] * up, y[3] * up),
                                    pack_e4m3x4(y[4] * up, y[5] * up, y[6] * up, y[7] * up)));
            if ((t & 15) == 0) {
                const int32_t kb = c / kFp8Block;
                uint8_t *const word = p.scales + ((int64_t)(kb >> 2) * p.R + row) * 4;
                word[kb & 3] = (uint8_t)e;
                if (kb == KB - 1)
                    for (int32_t b = (kb & 3) + 1; b < 4; ++b)
                        word[b] = 127;
            }
        }
    }
}

// A CTA (or each of its warps) takes rows in a stride of the grid and keeps its
// threads' share of dweight in registers; the CTAs' sums meet in `partials`,
// one row of C floats each, which column_sum_kernel adds in a fixed order.
template <int V, bool kWarpRow>
__global__ void __launch_bounds__(1024) rmsnorm_backward_kernel(const NormBackwardParams p)
{
    extern __shared__ float dw_smem[];  // warp rows: C floats
    __shared__ float red[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warps = (int)blockDim.x >> 5;
    const int T = kWarpRow ? 32 : (int)blockDim.x;
    const int t = kWarpRow ? (int)(threadIdx.x & 31u) : (int)threadIdx.x;
    const int64_t row0 = kWarpRow ? (int64_t)blockIdx.x * warps + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = kWarpRow ? (int64_t)gridDim.x * warps : gridDim.x;
    const bool vec = p.vec != 0;
    const int32_t C = p.C;
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.f;

    for (int64_t row = row0; row < p.R; row += step) {
        uint4 dv[V], hv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            dv[i] = load8_bf16(p.dy + row * p.lddy, (t + i * T) * 8, C, vec);
            hv[i] = load8_bf16(p.h + row * p.ldh, (t + i * T) * 8, C, vec);
        }
        const float rstd = p.rstd[row];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d[8], h[8], w[8];
            unpack8(dv[i], d);
            unpack8(hv[i], h);
            load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, vec, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = h[j] * rstd;
                dot = fmaf(d[j] * w[j], n, dot);
                dw[i][j] = fmaf(d[j], n, dw[i][j]);
            }
        }
        const float mean = row_sum<kWarpRow>(dot, red) / (float)C;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            if (c >= C)
                continue;
            float d[8], h[8], w[8], r[8];
            unpack8(dv[i], d);
            unpack8(hv[i], h);
            load8_weight(p.weight, p.w_fp32, c, C, vec, w);
            if (p.dres)
                unpack8(load8_bf16(p.dres + row * p.lddr, c, C, vec), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = rstd * (d[j] * w[j] - h[j] * rstd * mean);
                if (p.dres)
                    d[j] += r[j];
            }
            store8_bf16(p.dx + row * p.lddx, c, C, vec,
                        make_uint4(bf16_pair(d[0], d[1]), bf16_pair(d[2], d[3]), bf16_pair(d[4], d[5]),
                                   bf16_pair(d[6], d[7])));
        }
    }

    float *const out = p.partials + (int64_t)blockIdx.x * C;
    if constexpr (kWarpRow) {
        // the warps add their sums one after another
        for (int k = 0; k < warps; ++k) {
            if ((int)(threadIdx.x >> 5) == k) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int32_t c = (t + i * T) * 8 + j;
                        if (c < C) {
                            const float v = k == 0 ? dw[i][j] : dw_smem[c] + dw[i][j];
                            if (k == warps - 1)
                                out[c] = v;
                            else
                                dw_smem[c] = v;
                        }
                    }
            }
            __syncthreads();
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((t + i * T) * 8 + j < C)
                    out[(t + i * T) * 8 + j] = dw[i][j];
    }
}

constexpr int kSumRows = 16;

// dw[c] = sum of n rows of partials, 32 columns and kSumRows strands a CTA.
__global__ void __launch_bounds__(32 * kSumRows) column_sum_kernel(const float *partials, int32_t n, int32_t C,
                                                                   float *dw)
{
    __shared__ float red[kSumRows][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int32_t c = (int32_t)blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < C)
        for (int32_t g = y; g < n; g += kSumRows)
            s += partials[(int64_t)g * C + c];
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && c < C) {
#pragma unroll
        for (int k = 1; k < kSumRows; ++k)
            s += red[k][x];
        dw[c] = s;
    }
}

template <typename... Params>
cudaError_t launch(void (*fn)(Params...), int64_t grid, int threads, size_t smem, cudaStream_t stream, Params... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// How a row of C columns is shared out: a warp a row up to 1024 columns, else
// a CTA a row with `threads` threads, V vectors of 8 columns to a thread.
struct RowSplit {
    bool warp_row;
    int threads;
    int V;
};

RowSplit split_row(int64_t C, int max_v)
{
    const int64_t nv = (C + 7) / 8;
    if (nv <= 32 * max_v && nv <= 128)
        return {true, 128, nv <= 32 ? 1 : (nv <= 64 ? 2 : 4)};
    int V = 1;
    while (V < 4 && (nv + V - 1) / V > 1024)
        V *= 2;
    while (V < max_v && (nv + V - 1) / V > 256)
        V *= 2;
    return {false, (int)(((nv + V - 1) / V + 31) / 32 * 32), V};
}

template <bool kWarpRow, bool kRes>
auto norm_fn(int V)
{
    return V == 1 ? &rmsnorm_kernel<1, kWarpRow, kRes>
                  : (V == 2 ? &rmsnorm_kernel<2, kWarpRow, kRes> : &rmsnorm_kernel<4, kWarpRow, kRes>);
}

template <bool kWarpRow>
auto norm_backward_fn(int V)
{
    return V == 1 ? &rmsnorm_backward_kernel<1, kWarpRow>
                  : (V == 2 ? &rmsnorm_backward_kernel<2, kWarpRow> : &rmsnorm_backward_kernel<4, kWarpRow>);
}

}  // namespace

int launch_rmsnorm(const NormParams &p, int num_sms, cudaStream_t stream)
{
    // few rows: more threads a row, for latency; many: 4 vectors a thread
    const RowSplit s = split_row(p.C, p.R <= 2 * num_sms ? 1 : 4);
    const int64_t grid = s.warp_row ? ((int64_t)p.R + 3) / 4 : p.R;
    auto fn = s.warp_row ? (p.residual ? norm_fn<true, true>(s.V) : norm_fn<true, false>(s.V))
                         : (p.residual ? norm_fn<false, true>(s.V) : norm_fn<false, false>(s.V));
    return launch(fn, grid, s.threads, 0, stream, p);
}

int rmsnorm_backward_ctas(int64_t R, int64_t C, int num_sms)
{
    const RowSplit s = split_row(C, 2);
    const int64_t rows = s.warp_row ? (R + 3) / 4 : R;
    const int64_t most = (int64_t)num_sms * (s.threads >= 1024 ? 1 : 1024 / s.threads);
    return (int)(rows < most ? rows : most);
}

int launch_rmsnorm_backward(const NormBackwardParams &p, int num_sms, cudaStream_t stream)
{
    const RowSplit s = split_row(p.C, 2);
    const int grid = rmsnorm_backward_ctas(p.R, p.C, num_sms);
    auto fn = s.warp_row ? norm_backward_fn<true>(s.V) : norm_backward_fn<false>(s.V);
    const size_t smem = s.warp_row ? (size_t)p.C * sizeof(float) : 0;
    cudaError_t rc = launch(fn, grid, s.threads, smem, stream, p);
    if (rc != cudaSuccess)
        return rc;
    return launch(&column_sum_kernel, ((int64_t)p.C + 31) / 32, 32 * kSumRows, 0, stream,
                  (const float *)p.partials, (int32_t)grid, p.C, p.dw);
}

}  // namespace wstma
