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
//
// Memory-bound by its bytes (2 or 4 read, 1 or 2 written per element) only if it
// spends few instructions an element.  So bf16 input stays packed in pairs: a
// power of two scales it exactly in bf16, and maxima and products take one
// instruction for two elements.  Scales are found with integer arithmetic on the
// maximum's bits.  8192 x 8192 bf16: along the rows 31 us, 6.5 TB/s; both ways 47 us,
// 5.7 TB/s; both ways with one scale a tile 42 us, 6.4 TB/s, HBM-bound; along the columns
// 37 us, 5.4 TB/s, and with both factors, whose products are taken in fp32 wherever an
// element is used, 56 us, 3.6 TB/s.  6143 x 5999
// both ways, no row aligned: 34 us, 4.4 TB/s, by the shifts' instructions.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8_format.cuh"
#include "fp8_kernels.h"
#include "ptx.cuh"

namespace wstma {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t abs_bf16x2(uint32_t a)
{
    uint32_t r;
    asm("abs.bf16x2 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Both halves of a pair: infinities become NaN.
__device__ __forceinline__ uint32_t inf_to_nan_bf16x2(uint32_t w)
{
    if ((w & 0x7FFFu) == 0x7F80u)
        w |= 0x7Fu;
    if ((w & 0x7FFF0000u) == 0x7F800000u)
        w |= 0x7F0000u;
    return w;
}

// How a thread holds its 8 x 8 elements: bf16 pairs along the row; the same with
// factors, applied in fp32 wherever a value is used (holding 64 products instead
// costs half the occupancy); fp32.
enum { kPairs = 0, kFactored = 1, kFloats = 2 };

template <int kMode>
struct Elements;

template <>
struct Elements<kPairs> {
    uint32_t v[8][4];

    // rm[i], cm[c]: packed maxima of row i (two strands) and columns 2c, 2c + 1
    __device__ __forceinline__ void maxima(uint32_t (&rm)[8], uint32_t (&cm)[4]) const
    {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            cm[c] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                a[c] = abs_bf16x2(v[i][c]);
                cm[c] = max_bf16x2(cm[c], a[c]);
            }
            // the zero keeps a strand of nothing but NaN from being NaN itself
            rm[i] = max_bf16x2(max_bf16x2(max_bf16x2(a[0], a[1]), max_bf16x2(a[2], a[3])), 0u);
        }
    }

    __device__ __forceinline__ void no_infinities()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[i][c] = inf_to_nan_bf16x2(v[i][c]);
    }

    // codes of row i, scaled by 2^(127 - e)
    __device__ __forceinline__ uint2 row_codes(int i, uint32_t e) const
    {
        const uint32_t s = (254u - e) << 7, up = s | (s << 16);
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            w[c] = mul_bf16x2(v[i][c], up);
        return make_uint2(pack_e4m3x4(bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])),
                          pack_e4m3x4(bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3])));
    }

    // codes of columns 2 c and 2 c + 1 down the rows
    __device__ __forceinline__ void column_codes(int c, uint32_t e0, uint32_t e1, uint2 &q0, uint2 &q1) const
    {
        const uint32_t up = ((254u - e0) << 7) | ((254u - e1) << 23);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = mul_bf16x2(v[i][c], up);
        q0 = make_uint2(pack_e4m3x4(bf16_lo(w[0]), bf16_lo(w[1]), bf16_lo(w[2]), bf16_lo(w[3])),
                        pack_e4m3x4(bf16_lo(w[4]), bf16_lo(w[5]), bf16_lo(w[6]), bf16_lo(w[7])));
        q1 = make_uint2(pack_e4m3x4(bf16_hi(w[0]), bf16_hi(w[1]), bf16_hi(w[2]), bf16_hi(w[3])),
                        pack_e4m3x4(bf16_hi(w[4]), bf16_hi(w[5]), bf16_hi(w[6]), bf16_hi(w[7])));
    }
};

// What the two fp32 forms share, over their at(i, j).
template <typename Self>
struct FloatElements {
    // maxima rounded to bf16 pairs would lose the fp32 value that decides the
    // scale, so these are fp32 bits: rm[i] of row i, cm[j] of column j
    __device__ __forceinline__ void maxima(uint32_t (&rm)[8], uint32_t (&cm)[8]) const
    {
        const Self &self = static_cast<const Self &>(*this);
        float c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float r = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = fabsf(self.at(i, j));
                r = fmaxf(r, a);
                c[j] = fmaxf(c[j], a);
            }
            rm[i] = __float_as_uint(r);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            cm[j] = __float_as_uint(c[j]);
    }

    __device__ __forceinline__ uint2 row_codes(int i, uint32_t e) const
    {
        const Self &self = static_cast<const Self &>(*this);
        const float up = scale_inverse(e);
        return make_uint2(
            pack_e4m3x4(self.at(i, 0) * up, self.at(i, 1) * up, self.at(i, 2) * up, self.at(i, 3) * up),
            pack_e4m3x4(self.at(i, 4) * up, self.at(i, 5) * up, self.at(i, 6) * up, self.at(i, 7) * up));
    }

    __device__ __forceinline__ uint2 one_column(int j, uint32_t e) const
    {
        const Self &self = static_cast<const Self &>(*this);
        const float up = scale_inverse(e);
        return make_uint2(
            pack_e4m3x4(self.at(0, j) * up, self.at(1, j) * up, self.at(2, j) * up, self.at(3, j) * up),
            pack_e4m3x4(self.at(4, j) * up, self.at(5, j) * up, self.at(6, j) * up, self.at(7, j) * up));
    }

    __device__ __forceinline__ void column_codes(int c, uint32_t e0, uint32_t e1, uint2 &q0, uint2 &q1) const
    {
        q0 = one_column(2 * c, e0);
        q1 = one_column(2 * c + 1, e1);
    }
};

template <>
struct Elements<kFloats> : FloatElements<Elements<kFloats>> {
    float y[8][8];

    __device__ __forceinline__ float at(int i, int j) const { return y[i][j]; }

    __device__ __forceinline__ void no_infinities()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[i][j] = inf_to_nan(y[i][j]);
    }
};

template <>
struct Elements<kFactored> : FloatElements<Elements<kFactored>> {
    uint32_t v[8][4];
    float rf[8], cf[8];

    __device__ __forceinline__ float at(int i, int j) const
    {
        return (j & 1 ? bf16_hi(v[i][j >> 1]) : bf16_lo(v[i][j >> 1])) * rf[i] * cf[j];
    }

    // an element whose product is infinite becomes NaN, and so does its product
    __device__ __forceinline__ void no_infinities()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (is_inf(at(i, j)))
                    v[i][j >> 1] |= j & 1 ? 0x7FFF0000u : 0x7FFFu;
    }
};

// Magnitudes (no NaN) order like their bits, so maxima travel as integers from here on.
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v)
{
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

__device__ __forceinline__ uint32_t half_warp_max_bf16x2(uint32_t v)
{
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        v = max_bf16x2(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
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

// a, b, c, d: rows of four bytes -> columns of four bytes.
__device__ __forceinline__ void transpose_bytes(uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d)
{
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    a = __byte_perm(ab0, cd0, 0x5410);
    b = __byte_perm(ab0, cd0, 0x7632);
    c = __byte_perm(ab1, cd1, 0x5410);
    d = __byte_perm(ab1, cd1, 0x7632);
}

__device__ __forceinline__ void load_column_factor(const QuantizeParams &p, int32_t c, float (&f)[8])
{
    if (!p.column_factor || c >= p.C) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = 1.f;
    } else if (p.column_fp32) {
        load8_float(static_cast<const float *>(p.column_factor), c, p.C, p.column_vec, f);
    } else {
        unpack8(load8_bf16(static_cast<const uint16_t *>(p.column_factor), c, p.C, p.column_vec), f);
    }
}

template <int kMode, bool kRows, bool kCols>
__global__ void __launch_bounds__(kThreads, kMode == kFloats ? 2 : 3) quantize_kernel(const QuantizeParams p)
{
    constexpr bool kPacked = kMode == kPairs;  // maxima as bf16 pairs, else as fp32
    // a warp's column maxima: bf16 of 128 columns (packed) or fp32
    __shared__ __align__(16) uint32_t colmax[kCols ? kThreads / 32 : 1][kPacked ? 64 : 128];
    __shared__ uint32_t tilemax[kThreads / 32];
    __shared__ __align__(16) uint8_t turned[kCols ? kFp8Block * kFp8Block : 16];
    grid_dependency_wait();
    grid_launch_dependents();
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4;
    const uint32_t col_tiles = (uint32_t)(p.C + kFp8Block - 1) / kFp8Block;
    const int32_t rb = (int32_t)(blockIdx.x / col_tiles), cb = (int32_t)(blockIdx.x % col_tiles);
    const int32_t r0 = rb * kFp8Block + g * 8, c0 = cb * kFp8Block + l * 8;
    const int32_t R = p.R, C = p.C;
    const bool full = (rb + 1) * (int64_t)kFp8Block <= R && (cb + 1) * (int64_t)kFp8Block <= C;

    Elements<kMode> y;
    if constexpr (kMode != kFloats) {
        const uint16_t *const x = static_cast<const uint16_t *>(p.x) + (int64_t)r0 * p.ldx;
        if (full && p.x_vec) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 q = *reinterpret_cast<const uint4 *>(x + i * p.ldx + c0);
                y.v[i][0] = q.x, y.v[i][1] = q.y, y.v[i][2] = q.z, y.v[i][3] = q.w;
            }
        } else if (full) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 q = load8_bf16_words(x + i * p.ldx + c0);
                y.v[i][0] = q.x, y.v[i][1] = q.y, y.v[i][2] = q.z, y.v[i][3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 q = load8_bf16_shifted(x + i * p.ldx, c0, C, r0 + i < R);
                y.v[i][0] = q.x, y.v[i][1] = q.y, y.v[i][2] = q.z, y.v[i][3] = q.w;
            }
        }
        if constexpr (kMode == kFactored) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y.rf[i] = p.row_factor && r0 + i < R ? p.row_factor[r0 + i] : 1.f;
            load_column_factor(p, c0, y.cf);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + i;
            if (r < R && c0 < C) {
                load8_float(static_cast<const float *>(p.x) + r * p.ldx, c0, C, p.x_vec, y.y[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y.y[i][j] = 0.f;
            }
        }
        if (p.row_factor) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = r0 + i < R ? p.row_factor[r0 + i] : 1.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y.y[i][j] *= f;
            }
        }
        if (p.column_factor) {
            float cf[8];
            load_column_factor(p, c0, cf);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y.y[i][j] *= cf[j];
        }
    }

    // Maxima pass over NaN.  An infinity shows in them: rare, and then the tile's
    // infinities become NaN and the maxima are those of its finite values.
    constexpr int kColWords = kPacked ? 4 : 8;
    uint32_t rm[8], cm[kColWords];
    y.maxima(rm, cm);
    bool inf = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        inf = inf || (kPacked ? (rm[i] & 0x7F800000u) == 0x7F800000u || (rm[i] & 0x7F80u) == 0x7F80u
                              : rm[i] == 0x7F800000u);
    if (kCols || p.tile ? __syncthreads_or(inf) : __any_sync(0xFFFFFFFFu, inf)) {
        y.no_infinities();
        y.maxima(rm, cm);
    }

    uint32_t re[8], ce[8];  // scale bytes of the thread's rows and columns
    if (p.tile) {
        uint32_t m = 0u;
        if constexpr (kPacked) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = i ? max_bf16x2(m, rm[i]) : rm[i];
            m = max(m & 0xFFFFu, m >> 16) << 16;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = max(m, rm[i]);
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0)
            tilemax[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k)
            m = max(m, tilemax[k]);
        const uint32_t e = scale_byte(__uint_as_float(m));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            re[i] = ce[i] = e;
    } else {
        if constexpr (kRows) {
            if constexpr (kPacked) {
                // two rows to a word: half the shuffles
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint32_t m = half_warp_max_bf16x2(
                        max_bf16x2(__byte_perm(rm[i], rm[i + 1], 0x5410), __byte_perm(rm[i], rm[i + 1], 0x7632)));
                    re[i] = scale_byte(bf16_lo(m));
                    re[i + 1] = scale_byte(bf16_hi(m));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    re[i] = scale_byte(__uint_as_float(half_warp_max(rm[i])));
            }
        }
        if constexpr (kCols) {
            const int warp = threadIdx.x >> 5;
#pragma unroll
            for (int c = 0; c < kColWords; ++c) {
                const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, cm[c], 16);
                cm[c] = kPacked ? max_bf16x2(cm[c], o) : max(cm[c], o);
            }
            if ((threadIdx.x & 16) == 0) {
#pragma unroll
                for (int c = 0; c < kColWords; c += 4)
                    *reinterpret_cast<uint4 *>(&colmax[warp][l * kColWords + c]) =
                        make_uint4(cm[c], cm[c + 1], cm[c + 2], cm[c + 3]);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kThreads / 32; ++k)
#pragma unroll
                for (int c = 0; c < kColWords; c += 4) {
                    const uint4 o = *reinterpret_cast<const uint4 *>(&colmax[k][l * kColWords + c]);
                    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        cm[c + d] = kPacked ? max_bf16x2(cm[c + d], w[d]) : max(cm[c + d], w[d]);
                }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ce[j] = scale_byte(kPacked ? (j & 1 ? bf16_hi(cm[j >> 1]) : bf16_lo(cm[j >> 1]))
                                           : __uint_as_float(cm[kPacked ? 0 : j]));
        }
    }

    // lane l < 8 of a half-warp stores the scale of its row l; group g < 8 that of column g
    const int32_t KB = (C + kFp8Block - 1) / kFp8Block, KBt = (R + kFp8Block - 1) / kFp8Block;
    if constexpr (kRows) {
        uint32_t e = re[0];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            e = l == i ? re[i] : e;
        if (l < 8 && r0 + l < R)
            store_scale(p.scales, R, r0 + l, cb, KB, e);
    }
    if constexpr (kCols) {
        uint32_t e = ce[0];
#pragma unroll
        for (int j = 1; j < 8; ++j)
            e = g == j ? ce[j] : e;
        if (g < 8 && c0 + g < C)
            store_scale(p.scales_t, C, c0 + g, rb, KBt, e);
    }

    uint8_t *const turn = turned + ((g ^ l) << 3) + l * 8 * kFp8Block;  // + j * kFp8Block: column j
    if (kRows && kCols && p.tile) {
        // one scale: the row codes are the column codes, turned 4 x 4 bytes at a time
        uint2 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[i] = y.row_codes(i, re[0]);
            if (full)
                *reinterpret_cast<uint2 *>(p.codes + (int64_t)(r0 + i) * p.ldq + c0) = q[i];
            else if (r0 + i < R && c0 < C)
                store8_codes(p.codes + (int64_t)(r0 + i) * p.ldq, c0, C, q[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            transpose_bytes(q[i].x, q[i + 1].x, q[i + 2].x, q[i + 3].x);
            transpose_bytes(q[i].y, q[i + 1].y, q[i + 2].y, q[i + 3].y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<uint2 *>(turn + j * kFp8Block) = make_uint2(q[j].x, q[4 + j].x);
            *reinterpret_cast<uint2 *>(turn + (4 + j) * kFp8Block) = make_uint2(q[j].y, q[4 + j].y);
        }
    } else {
        if constexpr (kRows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint2 q = y.row_codes(i, re[i]);
                if (full)
                    *reinterpret_cast<uint2 *>(p.codes + (int64_t)(r0 + i) * p.ldq + c0) = q;
                else if (r0 + i < R && c0 < C)
                    store8_codes(p.codes + (int64_t)(r0 + i) * p.ldq, c0, C, q);
            }
        }
        if constexpr (kCols) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint2 q0, q1;
                y.column_codes(c, ce[2 * c], ce[2 * c + 1], q0, q1);
                *reinterpret_cast<uint2 *>(turn + 2 * c * kFp8Block) = q0;
                *reinterpret_cast<uint2 *>(turn + (2 * c + 1) * kFp8Block) = q1;
            }
        }
    }
    if constexpr (kCols) {
        // row c of the turned tile: 16 units of 8 bytes, unit u at u ^ (c / 8); the
        // half-warp g writes its rows 8 g .. 8 g + 7, 8 bytes a lane
        __syncthreads();
        const int32_t rl = rb * kFp8Block + l * 8;
        const int64_t cg = (int64_t)cb * kFp8Block + g * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint2 q = *reinterpret_cast<const uint2 *>(turned + (g * 8 + i) * kFp8Block + ((l ^ g) << 3));
            if (full)
                *reinterpret_cast<uint2 *>(p.codes_t + (cg + i) * p.ldqt + rl) = q;
            else if (cg + i < C && rl < R)
                store8_codes(p.codes_t + (cg + i) * p.ldqt, rl, R, q);
        }
    }
}

template <int kMode>
auto quantize_fn(bool rows, bool cols)
{
    return rows ? (cols ? &quantize_kernel<kMode, true, true> : &quantize_kernel<kMode, true, false>)
                : &quantize_kernel<kMode, false, true>;
}

}  // namespace

int launch_quantize(const QuantizeParams &p, cudaStream_t stream)
{
    const bool rows = p.codes != nullptr, cols = p.codes_t != nullptr;
    auto fn = p.x_fp32 ? quantize_fn<kFloats>(rows, cols)
                       : (p.row_factor || p.column_factor ? quantize_fn<kFactored>(rows, cols)
                                                          : quantize_fn<kPairs>(rows, cols));
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
