// Residual addition, root-mean-square norm and 8-bit quantisation in one pass,
// and the norm's gradients.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

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

// Sum over the threads of a row: the warp's when the row is a warp's, else the CTA's,
// which may have more rows after this one (kAgain).
template <bool kWarpRow, bool kAgain>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = warp_sum(v);
    if constexpr (kWarpRow) {
        return v;
    } else {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = (int)blockDim.x >> 5;
        if constexpr (kAgain)
            __syncthreads();  // the previous row's sums have been read
        if (lane == 0)
            red[warp] = v;
        __syncthreads();
        return warp_sum(lane < n ? red[lane] : 0.f);
    }
}

__device__ __forceinline__ void load8_weight(const void *w, int fp32, int32_t c, int32_t C, bool vec, uint64_t (&f)[4])
{
    if (fp32) {
        float g[8];
        load8_float(static_cast<const float *>(w), c, C, vec, g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[j] = f32x2(g[2 * j], g[2 * j + 1]);
    } else {
        unpack8_pairs(load8_bf16(static_cast<const uint16_t *>(w), c, C, vec), f);
    }
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

// How a row's bf16 arrays lie: 16-byte aligned; x, residual and h shifted alike (an
// odd number of columns in each); or each in its own way.
enum { kRowsAligned = 0, kRowsAlike = 1, kRowsAnyhow = 2 };

__device__ __forceinline__ uint4 add_bf16(uint4 x, uint4 r)
{
    float a[8], b[8];
    unpack8(x, a);
    unpack8(r, b);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        a[j] += b[j];
    return make_uint4(bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(a[4], a[5]), bf16_pair(a[6], a[7]));
}

__device__ __forceinline__ void add_squares(uint4 h, uint64_t &sum)
{
    uint64_t a[4];
    unpack8_pairs(h, a);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sum = fma_f32x2(a[j], a[j], sum);
}

__device__ __forceinline__ float both(uint64_t v)
{
    float lo, hi;
    f32x2_parts(v, lo, hi);
    return lo + hi;
}

// The 16-byte group of a row that starts `first` elements into it (less than 0, or
// reaching past C, at its ends), with zeros for what is not the row's; groups
// without any of it are not read.
__device__ __forceinline__ uint4 load_group(const uint16_t *row, int32_t first, int32_t C)
{
    if (first >= C)
        return make_uint4(0u, 0u, 0u, 0u);
    uint4 q = *reinterpret_cast<const uint4 *>(row + first);
    if (first < 0 || first + 8 > C) {
        uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (first + j < 0 || first + j >= C)
                w[j >> 1] &= j & 1 ? 0xFFFFu : 0xFFFF0000u;
        q = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return q;
}

__device__ __forceinline__ void store_group(uint16_t *row, int32_t first, int32_t C, uint4 q)
{
    if (first >= 0 && first + 8 <= C) {
        *reinterpret_cast<uint4 *>(row + first) = q;
        return;
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (first + j >= 0 && first + j < C)
            row[first + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}

// Largest of the half-warp's 16 lanes for each of V values, of which lane l is left
// with number l % V: lanes trade the values they do not keep, so that V maxima
// together take 3 + V exchanges at most and not 4 V.
template <int V>
__device__ __forceinline__ float half_warp_max(const float (&a)[V])
{
    const int lane = (int)threadIdx.x;
    float m = a[0];
    if constexpr (V >= 2) {
        const bool odd = lane & 1;
        m = fmaxf(odd ? a[1] : a[0], __shfl_xor_sync(0xFFFFFFFFu, odd ? a[0] : a[1], 1));
        if constexpr (V == 4) {
            const float n = fmaxf(odd ? a[3] : a[2], __shfl_xor_sync(0xFFFFFFFFu, odd ? a[2] : a[3], 1));
            const bool high = lane & 2;
            m = fmaxf(high ? n : m, __shfl_xor_sync(0xFFFFFFFFu, high ? m : n, 2));
        }
    }
#pragma unroll
    for (int d = V; d < 16; d *= 2)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    return m;
}

// A row's vectors t, t + T, ..., normalised and quantised: the maxima of a thread's
// V blocks are found, turned into scales and stored together (one by one, with more
// instructions, 8192 x 8192 without a residual takes 50 us; this way 44).
template <int V>
__device__ __forceinline__ void normalise(const NormParams &p, int64_t row, int t, int T, const uint4 (&h)[V],
                                          float rstd)
{
    const int32_t C = p.C;
    const uint64_t rstd2 = f32x2(rstd, rstd);
    uint64_t y[V][4];
    float amax[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        uint64_t w[4];
        unpack8_pairs(h[i], y[i]);
        load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, p.w_vec, w);
        amax[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[i][j] = mul_f32x2(mul_f32x2(y[i][j], rstd2), w[j]);
            float lo, hi;
            f32x2_parts(y[i][j], lo, hi);
            amax[i] = max3_abs(amax[i], lo, hi);
        }
    }
    float mine = half_warp_max<V>(amax);
    if (__any_sync(0xFFFFFFFFu, is_inf(mine))) {
        // a block with an infinity: its scale is that of its finite values
#pragma unroll
        for (int i = 0; i < V; ++i) {
            amax[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float lo, hi;
                f32x2_parts(y[i][j], lo, hi);
                amax[i] = fmaxf(amax[i], fmaxf(finite_abs(lo), finite_abs(hi)));
                y[i][j] = f32x2(inf_to_nan(lo), inf_to_nan(hi));
            }
        }
        mine = half_warp_max<V>(amax);
    }
    const uint32_t e = scale_byte(mine);
    const float inverse = scale_inverse(e);
    const int l = t & 15;
    if (l < V) {
        const int32_t KB = (C + kFp8Block - 1) / kFp8Block;
        const int32_t kb = (t + l * T) / 16;
        if (kb < KB) {
            uint8_t *const word = p.scales + ((int64_t)(kb >> 2) * p.R + row) * 4;
            word[kb & 3] = (uint8_t)e;
            if (kb == KB - 1)
                for (int32_t b = (kb & 3) + 1; b < 4; ++b)
                    word[b] = 127;
        }
    }
    uint8_t *const codes = p.codes + row * p.ldq;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int32_t c = (t + i * T) * 8;
        const float f = __shfl_sync(0xFFFFFFFFu, inverse, i, 16);
        const uint64_t up = f32x2(f, f);
        if (c < C)
            store8_codes(codes, c, C,
                         make_uint2(pack_e4m3x4(mul_f32x2(y[i][0], up), mul_f32x2(y[i][1], up)),
                                    pack_e4m3x4(mul_f32x2(y[i][2], up), mul_f32x2(y[i][3], up))));
    }
}

// One pass over the row, which stays in registers as bf16 (h is what is normalised,
// so nothing is lost): HBM-bound with a residual, 8192 x 8192 71 us, 6.6 TB/s; without
// one, 44 us and 4.6 TB/s, with no unit full: issue slots 58 % busy, DRAM 48 %, a warp
// waiting mostly for its loads with 29 of an SM's 64 warps there.
// Vector v of a row is its columns 8 v .. 8 v + 7: thread t of the row's T holds
// vectors t, t + T, ..., so the 16 lanes of a half-warp always hold one block of 128.
// Rows that are shifted alike are loaded, added and stored by 16-byte groups, and
// turned into vectors from two neighbouring lanes' groups; otherwise unaligned rows
// go vector by vector (5772 x 5391: 53 us, 69 that way).  Registers are capped at 64,
// for 1024 threads an SM, or 48 where two vectors a thread fit them (8192 x 4096 with
// a residual: 38 us, 41 with 50 registers).
template <int V, bool kWarpRow, bool kRes, int kRows>
__global__ void __maxnreg__(V == 2 && kRows == kRowsAligned ? 48 : 64) rmsnorm_kernel(const NormParams p)
{
    __shared__ float red[32];
    constexpr bool vec = kRows == kRowsAligned;
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
    uint64_t sum2 = 0u;
    float sum;
    if constexpr (kRows == kRowsAlike) {
        const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(xr) & 15u);
        const int32_t back = (int32_t)(mis >> 1);  // elements of the first group before the row
#pragma unroll
        for (int i = 0; i < V; ++i)
            hv[i] = load_group(xr, (t + i * T) * 8 - back, C);
        if constexpr (kRes) {
            uint4 rv[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                rv[i] = load_group(rr, (t + i * T) * 8 - back, C);
#pragma unroll
            for (int i = 0; i < V; ++i)
                hv[i] = add_bf16(hv[i], rv[i]);
        }
        // A vector's rest is in the next lane's group; a warp's last lane finds it
        // in shared memory, where each warp leaves its first lane's.
        __shared__ uint4 edge[kWarpRow ? 1 : V][kWarpRow ? 1 : 32];
        const int warp = t >> 5, lane = t & 31;
        if constexpr (!kWarpRow) {
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    edge[i][warp] = hv[i];
            }
            __syncthreads();
        }
        uint4 group[V];
        // by whole words, a case each (the row's is the same for all its threads), and
        // half a word: only the words that a shift needs are exchanged
        auto turn = [&](auto words) {
            constexpr int kWords = decltype(words)::value;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                group[i] = hv[i];
                uint4 right = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (kWarpRow) {
                    if (i + 1 < V)
                        right = hv[i + 1 < V ? i + 1 : i];
                } else {
                    const bool end = (warp + 1) * 32 == T;
                    if (!end || i + 1 < V)
                        right = edge[end ? (i + 1 < V ? i + 1 : i) : i][end ? 0 : warp + 1];
                }
                const uint32_t last[4] = {right.x, right.y, right.z, right.w};
                uint32_t w[8] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w};
#pragma unroll
                for (int k = 0; k <= kWords; ++k) {
                    if constexpr (kWarpRow) {
                        w[4 + k] = __shfl_sync(0xFFFFFFFFu, lane == 0 ? last[k] : w[k], (lane + 1) & 31);
                    } else {
                        const uint32_t n = __shfl_down_sync(0xFFFFFFFFu, w[k], 1);
                        w[4 + k] = lane == 31 ? last[k] : n;
                    }
                }
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = __funnelshift_r(w[kWords + k], w[kWords + k + 1], (mis & 2u) * 8u);
                hv[i] = make_uint4(o[0], o[1], o[2], o[3]);  // zeros stand past the row's end already
                add_squares(hv[i], sum2);
            }
        };
        switch (mis >> 2) {
        case 0: turn(std::integral_constant<int, 0>{}); break;
        case 1: turn(std::integral_constant<int, 1>{}); break;
        case 2: turn(std::integral_constant<int, 2>{}); break;
        default: turn(std::integral_constant<int, 3>{}); break;
        }
        sum = row_sum<kWarpRow, false>(both(sum2), red);
        // h may be x or residual: stored after every thread's loads
        if constexpr (kRes) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int32_t first = (t + i * T) * 8 - back;
                if (first < C)
                    store_group(p.h + row * p.ldh, first, C, group[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            hv[i] = load8_row(xr, (t + i * T) * 8, C, vec);
        if constexpr (kRes) {
            uint4 rv[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                rv[i] = load8_row(rr, (t + i * T) * 8, C, vec);
#pragma unroll
            for (int i = 0; i < V; ++i)
                hv[i] = add_bf16(hv[i], rv[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            add_squares(hv[i], sum2);
            if constexpr (kRes)
                store8_row(p.h + row * p.ldh, (t + i * T) * 8, C, vec, hv[i]);
        }
        sum = row_sum<kWarpRow, false>(both(sum2), red);
    }
    const float rstd = __frsqrt_rn(sum * p.inv_c + p.eps);
    if (p.rstd && t == 0)
        p.rstd[row] = rstd;
    if constexpr (V == 4 && kRows != kRowsAligned) {
        // two and two: the shifts leave no registers for four (6606 x 6634: 71 us, 74 with
        // four; aligned rows take 4 together: 8192 x 8192 71.2, 71.7 with two and two)
        const uint4 first[2] = {hv[0], hv[1]}, second[2] = {hv[2], hv[3]};
        normalise<2>(p, row, t, T, first, rstd);
        normalise<2>(p, row, t + 2 * T, T, second, rstd);
    } else {
        normalise<V>(p, row, t, T, hv, rstd);
    }
}

// The sums over 8 elements, two at a time: dot += dy w n, dw += dy n with n = h rstd.
__device__ __forceinline__ void backward_sums(uint4 dy, uint4 h, const uint64_t (&w)[4], uint64_t rstd2, uint64_t &dot,
                                              uint64_t (&dw)[4])
{
    uint64_t d[4], x[4];
    unpack8_pairs(dy, d);
    unpack8_pairs(h, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t n = mul_f32x2(x[j], rstd2);
        dot = fma_f32x2(mul_f32x2(d[j], w[j]), n, dot);
        dw[j] = fma_f32x2(d[j], n, dw[j]);
    }
}

// The gradient of 8 elements: rstd (dy w - n mean) + dresidual.
template <bool kDres>
__device__ __forceinline__ uint4 backward_values(uint4 dy, uint4 h, const uint64_t (&w)[4], uint4 dres, uint64_t rstd2,
                                                 uint64_t minus_mean2)
{
    uint64_t d[4], x[4], r[4];
    unpack8_pairs(dy, d);
    unpack8_pairs(h, x);
    if constexpr (kDres)
        unpack8_pairs(dres, r);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        d[j] = fma_f32x2(mul_f32x2(x[j], rstd2), minus_mean2, mul_f32x2(d[j], w[j]));
        if constexpr (kDres)
            d[j] = fma_f32x2(d[j], rstd2, r[j]);
        else
            d[j] = mul_f32x2(d[j], rstd2);
        float lo, hi;
        f32x2_parts(d[j], lo, hi);
        o[j] = bf16_pair(lo, hi);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sums of 8 columns as floats.
__device__ __forceinline__ void unpair8(const uint64_t (&v)[4], float (&f)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f32x2_parts(v[j], f[2 * j], f[2 * j + 1]);
}

constexpr int kBackwardThreads = 512;
constexpr int kRingMax = 64;               // slots of a CTA's rings of rows
constexpr int kRingBytes = 208 * 1024;     // of an SM's shared memory, shared by its CTAs

// Rows of more than four vectors a thread (C > 16384): a CTA takes rows in a stride of the
// grid and keeps its threads' share of dweight in registers.  The ring of the kernel below
// keeps the weights there too, and with eight vectors the two would take all of a
// thread's 128 registers; its memory would hold two rows up to C = 26624 (17749 with
// dresidual).  4096 x 20000 332 us, 2.0 TB/s; 2048 x 32768 219 us, 2.5 TB/s.
template <int V, bool kDres, bool kVec>
__global__ void __launch_bounds__(kBackwardThreads, 1) rmsnorm_backward_wide_kernel(const NormBackwardParams p)
{
    __shared__ float red[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int T = (int)blockDim.x, t = (int)threadIdx.x;
    const int32_t C = p.C;
    const float inv = 1.f / (float)C;
    uint64_t dw[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dw[i][j] = 0u;
    for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x) {
        uint4 dy[V], h[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            dy[i] = load8_row(p.dy + row * p.lddy, (t + i * T) * 8, C, kVec);
            h[i] = load8_row(p.h + row * p.ldh, (t + i * T) * 8, C, kVec);
        }
        const float rstd = p.rstd[row];
        const uint64_t rstd2 = f32x2(rstd, rstd);
        uint64_t dot = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint64_t w[4];
            load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, p.w_vec, w);
            backward_sums(dy[i], h[i], w, rstd2, dot, dw[i]);
        }
        const float mean = row_sum<false, true>(both(dot), red) * inv;
        const uint64_t minus_mean2 = f32x2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            uint64_t w[4];
            load8_weight(p.weight, p.w_fp32, c, C, p.w_vec, w);
            uint4 dres = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (kDres)
                dres = load8_row(p.dres + row * p.lddr, c, C, kVec);
            store8_row(p.dx + row * p.lddx, c, C, kVec,
                       backward_values<kDres>(dy[i], h[i], w, dres, rstd2, minus_mean2));
        }
    }
    float *const out = p.partials + (int64_t)blockIdx.x * C;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[8];
        unpair8(dw[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((t + i * T) * 8 + j < C)
                out[(t + i * T) * 8 + j] = f[j];
    }
}

// Eight elements from the 32 bytes at shared address `at`, which start kWords words
// (and half a word, `by` = 16 bits) into them.
template <int kWords>
__device__ __forceinline__ uint4 shifted_vector(uint32_t at, uint32_t by)
{
    uint32_t w[9], o[4];
    ld_shared_v4(at, w[0], w[1], w[2], w[3]);
    ld_shared_v4(at + 16u, w[4], w[5], w[6], w[7]);
    w[8] = 0u;  // of a shift by four words, which are whole
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = __funnelshift_r(w[kWords + k], w[kWords + k + 1], by);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A thread's vectors t, t + T, ... of a row whose bytes lie in shared memory at `at`,
// `mis` bytes into their first 16-byte group.  A case for each shift by whole words:
// `mis` is the same for all threads of a row.
template <int V, bool kVec>
__device__ __forceinline__ void ring_vectors(uint4 (&q)[V], uint32_t at, uint32_t mis, int t, int T, int32_t C)
{
    const uint32_t by = (mis & 2u) * 8u;
    auto read = [&](auto words) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            q[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < C)
                q[i] = shifted_vector<decltype(words)::value>(at + (uint32_t)c * 2u, by);
            if (c < C && c + 8 > C) {  // what follows the row is not its
                uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + 2 * k + 1 >= C)
                        w[k] = c + 2 * k < C ? w[k] & 0xFFFFu : 0u;
                q[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            q[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < C)
                ld_shared_v4(at + (uint32_t)c * 2u, q[i].x, q[i].y, q[i].z, q[i].w);
        }
    } else {
        switch (mis >> 2) {
        case 0: read(std::integral_constant<int, 0>{}); break;
        case 1: read(std::integral_constant<int, 1>{}); break;
        case 2: read(std::integral_constant<int, 2>{}); break;
        default: read(std::integral_constant<int, 3>{}); break;
        }
    }
}

// Stores the row that lies in shared memory 16 bytes behind `at` by the 16-byte groups
// of its place in global memory, of which there may be one more than it has vectors.
template <int V>
__device__ __forceinline__ void store_staged(uint16_t *row, uint32_t at, int t, int T, int32_t C)
{
    const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    const int32_t back = (int32_t)(mis >> 1);
    const uint32_t by = (mis & 2u) * 8u;
    auto write = [&](auto words) {
#pragma unroll
        for (int i = 0; i <= V; ++i) {
            const int32_t v = t + i * T, first = v * 8 - back;
            if (first < C)
                store_group(row, first, C, shifted_vector<decltype(words)::value>(at + (uint32_t)v * 16u, by));
        }
    };
    switch ((16u - mis) >> 2) {
    case 0: write(std::integral_constant<int, 0>{}); break;
    case 1: write(std::integral_constant<int, 1>{}); break;
    case 2: write(std::integral_constant<int, 2>{}); break;
    case 3: write(std::integral_constant<int, 3>{}); break;
    default: write(std::integral_constant<int, 4>{}); break;
    }
}

// A group of T threads (a multiple of 32) takes rows in a stride of all groups,
// `blockDim.x / T` groups to a CTA, and keeps its threads' share of dweight in
// registers.  Rows come through a ring of bulk copies in shared memory, slots of
// dy, h (and dresidual), so the bytes in flight are the ring's (up to 200 KB an SM)
// and not what the registers hold: that left HBM idle half of the time (6143 x
// 4104: 42 us with one row ahead in registers).  A group's first thread refills a
// slot after the barrier in the next row's reduction, which every thread reaches
// when it is done with the slot.  Rows that are not 16-byte aligned are copied
// with the rest of their first and last 16-byte groups, and their dx is left in shared
// memory, two rows of it, from which it is stored by 16-byte groups after that barrier
// (8000 x 4001 from 81 us, with lanes that exchange their vectors, to 65; with several
// groups to a CTA the exchange is as good, 5211 x 1363 23.5 us against 25.3).  The CTAs' sums meet in
// `partials`, one row of C floats each, which column_sum_kernel adds in a fixed
// order.
//
// HBM-bound where rows are aligned and long: 8192 x 8192 with dresidual 80.5 us, 6.7
// TB/s.  Four vectors a thread (C from 8193) read dy and h twice from shared memory, for
// their registers: 4096 x 8200 47 us, 127 without the ring; 4096 x 16384 99 us, 146
// without it (two slots leave gaps).  Short rows are bound by their instructions and
// the barrier in each: 8192 x 1024 19 us, 3.5 TB/s; 8000 x 1810 40 us, 2.9 TB/s.
template <int V, bool kDres, bool kVec, bool kGroups, int kThreads>
__global__ void __launch_bounds__(kThreads, V == 1 || kThreads <= 320 ? 2 : 1)
    rmsnorm_backward_ring_kernel(const NormBackwardParams p, const int32_t group_threads, const int32_t slots,
                                 const uint32_t pitch)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ __align__(8) uint64_t full[kRingMax];
    constexpr int kRows = kDres ? 3 : 2;
    constexpr bool kStage = !kVec && !kGroups && V <= 2;
    constexpr bool kHold = V <= 2;  // dy and h stay in registers between a row's two passes, else are read again
    const int T = kGroups ? group_threads : (int)blockDim.x;
    const int groups = kGroups ? (int)blockDim.x / T : 1, g = kGroups ? (int)threadIdx.x / T : 0;
    const int t = (int)threadIdx.x - g * T, lane = t & 31, warps = T >> 5;
    const int32_t C = p.C;
    const uint32_t slot_bytes = pitch * kRows;
    const uint32_t base = smem_u32(ring) + (uint32_t)(g * slots) * slot_bytes;
    const uint32_t bars = smem_u32(full) + 8u * (uint32_t)(g * slots);
    const uint32_t stage_bytes = pitch + 16u;
    const uint32_t staging = smem_u32(ring) + (uint32_t)(groups * slots) * slot_bytes + (uint32_t)g * 2u * stage_bytes;
    uint32_t staged = 0;  // which of the two
    const float inv = 1.f / (float)C;
    const uint32_t R = (uint32_t)p.R, step = gridDim.x * (uint32_t)groups;  // sums of rows fit 32 bits without a sign
    const uint32_t row0 = blockIdx.x * (uint32_t)groups + (uint32_t)g;
    if (t == 0) {
        for (int s = 0; s < slots; ++s)
            mbar_init(bars + 8u * s, 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    const uint16_t *const src[3] = {p.dy, p.h, p.dres};
    const int64_t ld[3] = {p.lddy, p.ldh, p.lddr};
    auto fill = [&](int s, uint32_t row) {
        const uint32_t bar = bars + 8u * s;
        uintptr_t from[kRows];
        uint32_t bytes[kRows], all = 0;
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            from[k] = reinterpret_cast<uintptr_t>(src[k] + row * ld[k]);
            const uint32_t end = ((uint32_t)(from[k] & 15u) + 2u * (uint32_t)C + 15u) & ~15u;
            bytes[k] = kVec ? 2u * (uint32_t)C : end;
            all += bytes[k];
        }
        mbar_arrive_expect_tx(bar, all);
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            bulk_load(base + (uint32_t)s * slot_bytes + (uint32_t)k * pitch,
                      reinterpret_cast<const void *>(from[k] & ~(uintptr_t)15), bytes[k], bar);
        }
    };
    auto mis = [&](int k, uint32_t row) {  // of the address, whose lowest bits need no more than 32
        return kVec ? 0u
                    : ((uint32_t)reinterpret_cast<uintptr_t>(src[k]) + 2u * row * (uint32_t)ld[k]) & 15u;
    };
    if (t == 0)
        for (int s = 0; s < slots && row0 + (uint32_t)s * step < R; ++s)
            fill(s, row0 + (uint32_t)s * step);

    uint64_t dw[V][4], w[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load8_weight(p.weight, p.w_fp32, (t + i * T) * 8, C, p.w_vec, w[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dw[i][j] = 0u;
    }
    float rstd = row0 < R ? p.rstd[row0] : 0.f;
    int s = 0;
    uint32_t ph = 0, buf = 0;
    bool ok = true;
    int before = -1;  // the slot of the row before, if a row is left for it
    for (uint32_t row = row0; row < R; row += step) {
        const float next_rstd = row + step < R ? p.rstd[row + step] : 0.f;
        // 2 s at most, and no more once that has run out
        ok = mbar_wait_tries(bars + 8u * s, ph, ok ? 10000000u : 1u, ok ? 200u : 1u) != 0u && ok;
        const uint32_t at = base + (uint32_t)s * slot_bytes;
        uint4 dy[kHold ? V : 1], h[kHold ? V : 1];
        const uint64_t rstd2 = f32x2(rstd, rstd);
        uint64_t dot2 = 0u;
        if constexpr (kHold) {
            ring_vectors<V, kVec>(dy, at, mis(0, row), t, T, C);
            ring_vectors<V, kVec>(h, at + pitch, mis(1, row), t, T, C);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (!kHold) {
                ring_vectors<1, kVec>(dy, at, mis(0, row), t + i * T, T, C);
                ring_vectors<1, kVec>(h, at + pitch, mis(1, row), t + i * T, T, C);
            }
            backward_sums(dy[kHold ? i : 0], h[kHold ? i : 0], w[i], rstd2, dot2, dw[i]);
        }
        // one barrier a row: the sums alternate between two buffers
        float dot = warp_sum(both(dot2));
        if (!kGroups || warps > 1) {
            float *const mine = red[buf] + g * warps;
            if (lane == 0)
                mine[t >> 5] = dot;
            if constexpr (kGroups)
                named_barrier_sync(1u + (uint32_t)g, (uint32_t)T);
            else
                __syncthreads();
            if constexpr (kGroups) {
                dot = 0.f;  // few warps: every lane adds their sums
                for (int k = 0; k < warps; ++k)
                    dot += mine[k];
            } else {
                dot = warp_sum(lane < warps ? mine[lane] : 0.f);
            }
            buf ^= 1u;
        } else {
            __syncwarp();
        }
        // not after a wait that ran out: a slot filled again before its copies have landed
        // would count an arrival too many into its barrier's phase, which faults
        if (t == 0 && before >= 0 && ok)
            fill(before, row + (uint32_t)(slots - 1) * step);
        if constexpr (kStage) {
            if (row != row0)
                store_staged<V>(p.dx + (int64_t)(row - step) * p.lddx, staging + (staged ^ 1u) * stage_bytes, t, T, C);
        }
        const uint64_t minus_mean2 = f32x2(-dot * inv, -dot * inv);
        uint4 dres[kHold ? V : 1];
        if constexpr (kDres && kHold)
            ring_vectors<V, kVec>(dres, at + 2u * pitch, mis(2, row), t, T, C);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            if constexpr (!kHold) {
                ring_vectors<1, kVec>(dy, at, mis(0, row), t + i * T, T, C);
                ring_vectors<1, kVec>(h, at + pitch, mis(1, row), t + i * T, T, C);
                if constexpr (kDres)
                    ring_vectors<1, kVec>(dres, at + 2u * pitch, mis(2, row), t + i * T, T, C);
            }
            const int v = kHold ? i : 0;
            const uint4 q = backward_values<kDres>(dy[v], h[v], w[i], dres[v], rstd2, minus_mean2);
            if constexpr (kStage) {
                if (c < C)
                    st_shared_v4(staging + staged * stage_bytes + 16u + 2u * (uint32_t)c, q.x, q.y, q.z, q.w);
            } else {
                store8_row(p.dx + (int64_t)row * p.lddx, c, C, kVec, q);
            }
        }
        staged ^= 1u;
        rstd = next_rstd;
        before = row + (uint32_t)slots * step < R ? s : -1;
        if (++s == slots) {
            s = 0;
            ph ^= 1u;
        }
    }
    if constexpr (kStage) {
        __syncthreads();
        if (row0 < R)
            store_staged<V>(p.dx + (int64_t)(row0 + (R - 1 - row0) / step * step) * p.lddx,
                            staging + (staged ^ 1u) * stage_bytes, t, T, C);
    }
    // a wait that ran out (its copies never landed): dweight says so
    if (!ok)
        dw[0][0] = f32x2(__int_as_float(0x7FFFFFFF), 0.f);

    float *const out = p.partials + (int64_t)blockIdx.x * C;
    float f[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
        unpair8(dw[i], f[i]);
    if constexpr (!kGroups && kVec) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t c = (t + i * T) * 8;
            if (c < C) {
                *reinterpret_cast<float4 *>(out + c) = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
                *reinterpret_cast<float4 *>(out + c + 4) = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
            }
        }
        return;
    }
    // the groups' sums meet in the ring, whose copies have all been used
    float *const sums = reinterpret_cast<float *>(ring);
    __syncthreads();
    if (g > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((t + i * T) * 8 + j < C)
                    sums[(g - 1) * C + (t + i * T) * 8 + j] = f[i][j];
    }
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int32_t c = (t + i * T) * 8 + j;
                if (c < C) {
                    float v = f[i][j];
                    for (int k = 0; k + 1 < groups; ++k)
                        v += sums[k * C + c];
                    out[c] = v;
                }
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

// V is 1, 2 or 4: the least that keeps a CTA within 1024 threads, then up to max_v
// while the CTA has more than 256.
RowSplit split_row(int64_t C, int max_v)
{
    const int64_t nv = (C + 7) / 8;
    if (nv <= 32 * max_v && nv <= 128)
        return {true, 128, nv <= 32 ? 1 : (nv <= 64 ? 2 : 4)};
    int V = 1;
    while ((nv + V - 1) / V > 1024)
        V *= 2;
    while (V < max_v && (nv + V - 1) / V > 256)
        V *= 2;
    return {false, (int)(((nv + V - 1) / V + 31) / 32 * 32), V};
}

template <bool kRes, int kRows>
auto norm_fn(const RowSplit &s)
{
    if (s.warp_row)
        return s.V == 1 ? &rmsnorm_kernel<1, true, kRes, kRows>
                        : (s.V == 2 ? &rmsnorm_kernel<2, true, kRes, kRows> : &rmsnorm_kernel<4, true, kRes, kRows>);
    return s.V == 1 ? &rmsnorm_kernel<1, false, kRes, kRows>
                    : (s.V == 2 ? &rmsnorm_kernel<2, false, kRes, kRows> : &rmsnorm_kernel<4, false, kRes, kRows>);
}

template <int kRows>
auto norm_fn(const NormParams &p, const RowSplit &s)
{
    return p.residual ? norm_fn<true, kRows>(s) : norm_fn<false, kRows>(s);
}

// Whether two row arrays are shifted alike in every row.
bool alike(const void *a, int64_t lda, const void *b, int64_t ldb)
{
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0 && (lda - ldb) % 8 == 0;
}

// How the gradient kernels share out rows of C columns: groups of T threads with V
// vectors each, `groups` to a CTA and `blocks` CTAs to an SM.
struct BackwardSplit {
    bool ring;
    int V, T, groups, blocks;
};

BackwardSplit split_backward(int64_t R, int64_t C, int num_sms)
{
    const int64_t nv = (C + 7) / 8;
    BackwardSplit s;
    s.V = 1;
    while ((nv + s.V - 1) / s.V > kBackwardThreads)
        s.V *= 2;
    s.T = (int)(((nv + s.V - 1) / s.V + 31) / 32 * 32);
    s.ring = s.V <= 4;
    s.groups = std::min(kBackwardThreads / s.T, s.T == 32 ? 16 : 15);  // barriers 1..15
    // few rows: on as many SMs as there are rows for
    s.groups = (int)std::min<int64_t>(s.groups, std::max<int64_t>(1, R / num_sms));
    s.blocks = s.V == 1 || (s.V == 2 && s.T <= 320) ? 2 : 1;
    return s;
}

template <bool kDres, bool kVec>
auto backward_ring_fn(const BackwardSplit &s)
{
    constexpr int kT = kBackwardThreads;
    if (s.groups > 1)
        return &rmsnorm_backward_ring_kernel<1, kDres, kVec, true, kT>;
    if (s.V == 4)
        return &rmsnorm_backward_ring_kernel<4, kDres, kVec, false, kT>;
    return s.V == 1 ? &rmsnorm_backward_ring_kernel<1, kDres, kVec, false, kT>
                    : (s.T <= 320 ? &rmsnorm_backward_ring_kernel<2, kDres, kVec, false, 320>
                                  : &rmsnorm_backward_ring_kernel<2, kDres, kVec, false, kT>);
}

// Rows of 8 vectors a thread end at 512 * 8 * 8 columns, the limit of the API.
static_assert(kBackwardThreads * 8 * 8 >= 32768, "every width up to the limit has a kernel");

}  // namespace

int launch_rmsnorm(const NormParams &p, int num_sms, cudaStream_t stream)
{
    // A row shifted by up to 7 elements may touch a group more than it has vectors;
    // 1024 threads of 4 hold 32768 columns.
    const int64_t span = (int64_t)p.C + 7;
    const bool same =
        !p.residual || (alike(p.x, p.ldx, p.residual, p.ldr) && alike(p.x, p.ldx, p.h, p.ldh));
    const int rows = p.vec ? kRowsAligned : (same && span <= 32768 ? kRowsAlike : kRowsAnyhow);
    // few rows: more threads a row, for latency; many: 4 vectors a thread
    const RowSplit s = split_row(rows == kRowsAlike ? span : p.C, p.R <= 2 * num_sms ? 1 : 4);
    const int64_t grid = s.warp_row ? ((int64_t)p.R + 3) / 4 : p.R;
    auto fn = rows == kRowsAligned ? norm_fn<kRowsAligned>(p, s)
                                   : (rows == kRowsAlike ? norm_fn<kRowsAlike>(p, s) : norm_fn<kRowsAnyhow>(p, s));
    return launch(fn, grid, s.threads, 0, stream, p);
}

int rmsnorm_backward_ctas(int64_t R, int64_t C, int num_sms)
{
    const BackwardSplit s = split_backward(R, C, num_sms);
    const int64_t ctas = (R + s.groups - 1) / s.groups;
    return (int)std::min<int64_t>(ctas, (int64_t)num_sms * s.blocks);
}

int launch_rmsnorm_backward(const NormBackwardParams &p, int num_sms, cudaStream_t stream)
{
    const BackwardSplit s = split_backward(p.R, p.C, num_sms);
    const int grid = rmsnorm_backward_ctas(p.R, p.C, num_sms);
    // whole 16-byte groups: plain vectors; else with room for the first and last group's rest
    const bool vec = p.vec && p.C % 8 == 0;
    cudaError_t rc;
    if (s.ring) {
        const int64_t pitch = vec ? (int64_t)p.C * 2 : ((int64_t)p.C * 2 + 15) / 16 * 16 + 16;
        const int64_t slot = pitch * (p.dres ? 3 : 2);
        const int64_t staging = vec || s.groups > 1 || s.V == 4 ? 0 : 2 * (pitch + 16);  // V = 4: room for two slots
        const int slots =
            (int)std::min<int64_t>((kRingBytes / s.blocks / s.groups - staging) / slot, kRingMax / s.groups);
        const int64_t sums = (int64_t)(s.groups - 1) * p.C * (int64_t)sizeof(float);
        auto fn = p.dres ? (vec ? backward_ring_fn<true, true>(s) : backward_ring_fn<true, false>(s))
                         : (vec ? backward_ring_fn<false, true>(s) : backward_ring_fn<false, false>(s));
        rc = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (rc == cudaSuccess)
            rc = launch(fn, grid, s.T * s.groups, (size_t)std::max<int64_t>((slots * slot + staging) * s.groups, sums), stream, p,
                        (int32_t)s.T, (int32_t)slots, (uint32_t)pitch);
    } else {
        auto fn = p.dres ? (vec ? &rmsnorm_backward_wide_kernel<8, true, true>
                                : &rmsnorm_backward_wide_kernel<8, true, false>)
                         : (vec ? &rmsnorm_backward_wide_kernel<8, false, true>
                                : &rmsnorm_backward_wide_kernel<8, false, false>);
        rc = launch(fn, grid, s.T, 0, stream, p);
    }
    if (rc != cudaSuccess)
        return rc;
    return launch(&column_sum_kernel, ((int64_t)p.C + 31) / 32, 32 * kSumRows, 0, stream,
                  (const float *)p.partials, (int32_t)grid, p.C, p.dw);
}

}  // namespace wstma
