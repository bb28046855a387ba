// Residual addition, root-mean-square norm and 8-bit quantisation in one pass,
// and the norm's gradients.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8_format.cuh"
#include "fp8_kernels.h"
#include "fp8_ptx.cuh"

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

// Rows that are not 16-byte aligned (an odd number of columns) go by aligned
// accesses and shifts, 8 columns a lane all the same.
__device__ __forceinline__ uint4 load8_row(const uint16_t *row, int32_t c, int32_t C, bool vec)
{
    return vec ? load8_bf16(row, c, C, true) : load8_bf16_shifted(row, c, C, true);
}

__device__ __forceinline__ void store8_row(uint16_t *row, int32_t c, int32_t C, bool vec, uint4 q)
{
    if (!vec)
        store8_bf16_shifted(row, c, C, c < C, q);
    else if (c < C)
        store8_bf16(row, c, C, true, q);
}

// Vector v of a row (8 columns each): thread t of the row's T holds vectors t,
// t + T, ..., so the 16 lanes of a half-warp always hold one block of 128.
template <int V, bool kWarpRow, bool kRes, bool vec>
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
    const int32_t C = p.C;
    const uint16_t *const xr = p.x + row * p.ldx;
    const uint16_t *const rr = kRes ? p.residual + row * p.ldr : nullptr;

    uint4 hv[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        hv[i] = load8_row(xr, (t + i * T) * 8, C, vec);
    if constexpr (kRes) {
        uint4 rv[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            rv[i] = load8_row(rr, (t + i * T) * 8, C, vec);
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
            store8_row(p.h + row * p.ldh, (t + i * T) * 8, C, vec, hv[i]);
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
        load8_weight(p.weight, p.w_fp32, c, C, p.w_vec, w);
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

// A row's share of one thread.
template <int V, bool kDres, bool kVec>
struct BackwardRow {
    uint4 dy[V], h[V], dres[kDres ? V : 1];
    float rstd;

    __device__ __forceinline__ void load(const NormBackwardParams &p, int64_t row, int t, int T)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            dy[i] = load8_row(p.dy + row * p.lddy, c, p.C, kVec);
            h[i] = load8_row(p.h + row * p.ldh, c, p.C, kVec);
            if constexpr (kDres)
                dres[i] = load8_row(p.dres + row * p.lddr, c, p.C, kVec);
        }
        rstd = p.rstd[row];
    }
};

constexpr int kBackwardThreads = 512;
constexpr int kRingMax = 32;               // slots of the ring of rows
constexpr int kRingBytes = 208 * 1024;     // of an SM's shared memory, shared by its CTAs

// A CTA (or each of its warps) takes rows in a stride of the grid and keeps its
// threads' share of dweight in registers; the CTAs' sums meet in `partials`,
// one row of C floats each, which column_sum_kernel adds in a fixed order.  Bound
// by HBM (4 to 8 bytes an element) if loads are always in flight: the next
// row's are issued before the current row's reduction (V <= 2, where the registers
// suffice).
//
// kThreads bounds the CTA: with V = 1, or up to 320 threads, two CTAs share an SM,
// so that one's reduction overlaps the other's loads and stores.
template <int V, bool kWarpRow, bool kDres, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, kWarpRow ? 6 : (V == 1 || kThreads <= 320 ? 2 : 1))
    rmsnorm_backward_kernel(const NormBackwardParams p)
{
    constexpr bool kAhead = V <= 2;
    extern __shared__ float dw_smem[];  // warp rows: C floats
    __shared__ float red[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warps = (int)blockDim.x >> 5;
    const int T = kWarpRow ? 32 : (int)blockDim.x;
    const int t = kWarpRow ? (int)(threadIdx.x & 31u) : (int)threadIdx.x;
    const int64_t row0 = kWarpRow ? (int64_t)blockIdx.x * warps + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = kWarpRow ? (int64_t)gridDim.x * warps : gridDim.x;
    const int32_t C = p.C;
    const float inv = 1.f / (float)C;
    float dw[V][8], w[kAhead ? V : 1][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.f;

    BackwardRow<V, kDres, kVec> cur, next;
    if (row0 < p.R)
        cur.load(p, row0, t, T);
    if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, p.w_vec, w[i]);
    }
    for (int64_t row = row0; row < p.R; row += step) {
        if constexpr (kAhead) {
            if (row + step < p.R)
                next.load(p, row + step, t, T);
        }
        const float rstd = cur.rstd;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d[8], h[8];
            unpack8(cur.dy[i], d);
            unpack8(cur.h[i], h);
            if constexpr (!kAhead)
                load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, p.w_vec, w[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = h[j] * rstd;
                dot = fmaf(d[j] * w[kAhead ? i : 0][j], n, dot);
                dw[i][j] = fmaf(d[j], n, dw[i][j]);
            }
        }
        const float mean = row_sum<kWarpRow>(dot, red) * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            float d[8], h[8], r[8];
            unpack8(cur.dy[i], d);
            unpack8(cur.h[i], h);
            if constexpr (!kAhead)
                load8_weight(p.weight, p.w_fp32, c, C, p.w_vec, w[0]);
            if constexpr (kDres)
                unpack8(cur.dres[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = rstd * (d[j] * w[kAhead ? i : 0][j] - h[j] * rstd * mean);
                if constexpr (kDres)
                    d[j] += r[j];
            }
            store8_row(p.dx + row * p.lddx, c, C, kVec,
                       make_uint4(bf16_pair(d[0], d[1]), bf16_pair(d[2], d[3]), bf16_pair(d[4], d[5]),
                                  bf16_pair(d[6], d[7])));
        }
        if constexpr (kAhead)
            cur = next;
        else if (row + step < p.R)
            cur.load(p, row + step, t, T);
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

// The same for rows that start and end at multiples of 16 bytes: rows come through
// a ring of bulk copies in shared memory, slots of dy, h (and dresidual), so the
// bytes in flight are the ring's (up to 200 KB an SM) and not what the registers
// hold: that left HBM idle half of the time (6143 x 4104: 42 us with one row ahead
// in registers).  Thread 0 refills a slot after the barrier in the next row's
// reduction, which every thread reaches when it is done with the slot.
template <int V, bool kDres, int kThreads>
__global__ void __launch_bounds__(kThreads, V == 1 || kThreads <= 320 ? 2 : 1)
    rmsnorm_backward_ring_kernel(const NormBackwardParams p, const int32_t slots)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ __align__(8) uint64_t full[kRingMax];
    constexpr int kRows = kDres ? 3 : 2;
    const int T = (int)blockDim.x, t = (int)threadIdx.x;
    const int warp = t >> 5, lane = t & 31, warps = T >> 5;
    const int32_t C = p.C;
    const uint32_t row_bytes = (uint32_t)C * 2u;
    const uint32_t slot_bytes = row_bytes * kRows;
    const uint32_t base = smem_u32(ring), bars = smem_u32(full);
    const float inv = 1.f / (float)C;
    const int64_t step = gridDim.x;
    if (t == 0) {
        for (int s = 0; s < slots; ++s)
            mbar_init(bars + 8u * s, 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    auto fill = [&](int s, int64_t row) {
        const uint32_t at = base + (uint32_t)s * slot_bytes, bar = bars + 8u * s;
        mbar_arrive_expect_tx(bar, slot_bytes);
        bulk_load(at, p.dy + row * p.lddy, row_bytes, bar);
        bulk_load(at + row_bytes, p.h + row * p.ldh, row_bytes, bar);
        if constexpr (kDres)
            bulk_load(at + 2u * row_bytes, p.dres + row * p.lddr, row_bytes, bar);
    };
    if (t == 0)
        for (int s = 0; s < slots && blockIdx.x + s * step < p.R; ++s)
            fill(s, blockIdx.x + s * step);

    float dw[V][8], w[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, p.w_vec, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.f;
    }
    float rstd = blockIdx.x < p.R ? p.rstd[blockIdx.x] : 0.f;
    int s = 0;
    uint32_t ph = 0, buf = 0;
    bool ok = true;
    int64_t refill = -1;  // row to load into the slot before this one
    int before = 0;
    for (int64_t row = blockIdx.x; row < p.R; row += step) {
        const float next_rstd = row + step < p.R ? p.rstd[row + step] : 0.f;
        ok = mbar_wait_tries(bars + 8u * s, ph, 10000000u, 200u) != 0u && ok;  // 2 s at most
        const uint32_t at = base + (uint32_t)s * slot_bytes;
        uint4 dy[V], h[V];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            dy[i] = h[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < C) {
                ld_shared_v4(at + (uint32_t)c * 2u, dy[i].x, dy[i].y, dy[i].z, dy[i].w);
                ld_shared_v4(at + row_bytes + (uint32_t)c * 2u, h[i].x, h[i].y, h[i].z, h[i].w);
            }
            float d[8], x[8];
            unpack8(dy[i], d);
            unpack8(h[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = x[j] * rstd;
                dot = fmaf(d[j] * w[i][j], n, dot);
                dw[i][j] = fmaf(d[j], n, dw[i][j]);
            }
        }
        // one barrier a row: the sums alternate between two buffers
        dot = warp_sum(dot);
        if (lane == 0)
            red[buf][warp] = dot;
        __syncthreads();
        if (t == 0 && refill >= 0)
            fill(before, refill);
        const float mean = warp_sum(lane < warps ? red[buf][lane] : 0.f) * inv;
        buf ^= 1u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            if (c >= C)
                continue;
            float d[8], x[8], r[8];
            unpack8(dy[i], d);
            unpack8(h[i], x);
            if constexpr (kDres) {
                uint4 q;
                ld_shared_v4(at + 2u * row_bytes + (uint32_t)c * 2u, q.x, q.y, q.z, q.w);
                unpack8(q, r);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = rstd * (d[j] * w[i][j] - x[j] * rstd * mean);
                if constexpr (kDres)
                    d[j] += r[j];
            }
            *reinterpret_cast<uint4 *>(p.dx + row * p.lddx + c) = make_uint4(
                bf16_pair(d[0], d[1]), bf16_pair(d[2], d[3]), bf16_pair(d[4], d[5]), bf16_pair(d[6], d[7]));
        }
        rstd = next_rstd;
        before = s;
        refill = row + slots * step < p.R ? row + slots * step : -1;
        if (++s == slots) {
            s = 0;
            ph ^= 1u;
        }
    }
    // a wait that ran out (its copies never landed): dweight says so
    const float poison = ok ? 0.f : __int_as_float(0x7FFFFFFF);
    float *const out = p.partials + (int64_t)blockIdx.x * C;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t c = (t + i * T) * 8;
        if (c < C) {
            *reinterpret_cast<float4 *>(out + c) =
                make_float4(dw[i][0] + poison, dw[i][1] + poison, dw[i][2] + poison, dw[i][3] + poison);
            *reinterpret_cast<float4 *>(out + c + 4) =
                make_float4(dw[i][4] + poison, dw[i][5] + poison, dw[i][6] + poison, dw[i][7] + poison);
        }
    }
}

constexpr int kSumRows = 32;

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
    if (c < C) {
#pragma unroll 8
        for (int32_t g = y; g < n; g += kSumRows)
            s += partials[(int64_t)g * C + c];
    }
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

// V is 1, 2, 4 or 8: the least that keeps a CTA within `most` threads, then up
// to max_v while the CTA has more than `wanted`.
RowSplit split_row(int64_t C, int max_v, int most, int wanted)
{
    const int64_t nv = (C + 7) / 8;
    if (nv <= 32 * max_v && nv <= 128)
        return {true, 128, nv <= 32 ? 1 : (nv <= 64 ? 2 : 4)};
    int V = 1;
    while ((nv + V - 1) / V > most)
        V *= 2;
    while (V < max_v && (nv + V - 1) / V > wanted)
        V *= 2;
    return {false, (int)(((nv + V - 1) / V + 31) / 32 * 32), V};
}

template <bool kRes, bool kVec>
auto norm_fn(const RowSplit &s)
{
    if (s.warp_row)
        return s.V == 1 ? &rmsnorm_kernel<1, true, kRes, kVec>
                        : (s.V == 2 ? &rmsnorm_kernel<2, true, kRes, kVec> : &rmsnorm_kernel<4, true, kRes, kVec>);
    return s.V == 1 ? &rmsnorm_kernel<1, false, kRes, kVec>
                    : (s.V == 2 ? &rmsnorm_kernel<2, false, kRes, kVec> : &rmsnorm_kernel<4, false, kRes, kVec>);
}

template <bool kDres, bool kVec>
auto norm_backward_fn(const RowSplit &s)
{
    constexpr int kT = kBackwardThreads;
    if (s.warp_row)
        return s.V == 1 ? &rmsnorm_backward_kernel<1, true, kDres, kVec, 128>
                        : &rmsnorm_backward_kernel<2, true, kDres, kVec, 128>;
    switch (s.V) {
    case 1: return &rmsnorm_backward_kernel<1, false, kDres, kVec, kT>;
    case 2:
        return s.threads <= 320 ? &rmsnorm_backward_kernel<2, false, kDres, kVec, 320>
                                : &rmsnorm_backward_kernel<2, false, kDres, kVec, kT>;
    case 4: return &rmsnorm_backward_kernel<4, false, kDres, kVec, kT>;
    default: return &rmsnorm_backward_kernel<8, false, kDres, kVec, kT>;
    }
}

// Rows of 8 vectors a thread end at 512 * 8 * 8 columns, the limit of the API.
static_assert(kBackwardThreads * 8 * 8 >= 32768, "every width up to the limit has a kernel");

}  // namespace

int launch_rmsnorm(const NormParams &p, int num_sms, cudaStream_t stream)
{
    // few rows: more threads a row, for latency; many: 4 vectors a thread
    const RowSplit s = split_row(p.C, p.R <= 2 * num_sms ? 1 : 4, 1024, 256);
    const int64_t grid = s.warp_row ? ((int64_t)p.R + 3) / 4 : p.R;
    auto fn = p.residual ? (p.vec ? norm_fn<true, true>(s) : norm_fn<true, false>(s))
                         : (p.vec ? norm_fn<false, true>(s) : norm_fn<false, false>(s));
    return launch(fn, grid, s.threads, 0, stream, p);
}

// CTAs of the gradient kernel on an SM: the bounds of the kernels' registers.
int backward_blocks(const RowSplit &s)
{
    if (s.warp_row)
        return 6;
    return s.V == 1 ? std::min(kBackwardThreads / s.threads * 2, 8) : (s.V == 2 && s.threads <= 320 ? 2 : 1);
}

int rmsnorm_backward_ctas(int64_t R, int64_t C, int num_sms)
{
    const RowSplit s = split_row(C, 2, kBackwardThreads, kBackwardThreads);
    const int64_t rows = s.warp_row ? (R + 3) / 4 : R;
    const int64_t most = (int64_t)num_sms * backward_blocks(s);
    return (int)(rows < most ? rows : most);
}

template <bool kDres>
auto norm_backward_ring_fn(const RowSplit &s)
{
    constexpr int kT = kBackwardThreads;
    return s.V == 1 ? &rmsnorm_backward_ring_kernel<1, kDres, kT>
                    : (s.threads <= 320 ? &rmsnorm_backward_ring_kernel<2, kDres, 320>
                                        : &rmsnorm_backward_ring_kernel<2, kDres, kT>);
}

int launch_rmsnorm_backward(const NormBackwardParams &p, int num_sms, cudaStream_t stream)
{
    const RowSplit s = split_row(p.C, 2, kBackwardThreads, kBackwardThreads);
    const int grid = rmsnorm_backward_ctas(p.R, p.C, num_sms);
    auto fn = p.dres ? (p.vec ? norm_backward_fn<true, true>(s) : norm_backward_fn<true, false>(s))
                     : (p.vec ? norm_backward_fn<false, true>(s) : norm_backward_fn<false, false>(s));
    const size_t smem = s.warp_row ? (size_t)p.C * sizeof(float) : 0;
    // the ring where rows are whole 16-byte groups and two or more slots fit
    const int64_t slot = (int64_t)p.C * 2 * (p.dres ? 3 : 2);
    const int64_t slots = std::min<int64_t>(kRingBytes / backward_blocks(s) / slot, kRingMax);
    cudaError_t rc;
    if (p.vec && p.C % 8 == 0 && !s.warp_row && s.V <= 2 && slots >= 2) {
        auto ring = p.dres ? norm_backward_ring_fn<true>(s) : norm_backward_ring_fn<false>(s);
        rc = cudaFuncSetAttribute(ring, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (rc == cudaSuccess)
            rc = launch(ring, grid, s.threads, (size_t)(slots * slot), stream, p, (int32_t)slots);
    } else {
        rc = launch(fn, grid, s.threads, smem, stream, p);
    }
    if (rc != cudaSuccess)
        return rc;
    return launch(&column_sum_kernel, ((int64_t)p.C + 31) / 32, 32 * kSumRows, 0, stream,
                  (const float *)p.partials, (int32_t)grid, p.C, p.dw);
}

}  // namespace wstma
