// The 8-bit block format: e4m3 codes with one power-of-two scale per block of
// 128, shared by the quantiser and the norm.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace wstma {

constexpr int kFp8Block = 128;

// Biased exponent of the least power of two s with amax / s <= 448.  448 is
// 1.75 * 2^8, so amax = m * 2^E with m in [1, 2) needs 2^(E-8) where m <= 1.75
// and 2^(E-7) above: integer arithmetic on the bits, exact for every finite
// amax.  Subnormal amax (and zero) ends at the least scale, 2^-127.
__device__ __forceinline__ uint32_t scale_byte(float amax)
{
    // a mantissa above 0.75 carries into the exponent
    const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
    return (uint32_t)max(e, 0);
}

// 1 / 2^(byte - 127), a normal number for every byte scale_byte() gives (<= 247).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two values -> two e4m3 codes, round to nearest even; `lo` lands in the low
// byte.  Inputs are at most 448 in magnitude, or NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d)
{
    return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

__device__ __forceinline__ bool is_inf(float f) { return (__float_as_uint(f) & 0x7FFFFFFFu) == 0x7F800000u; }

__device__ __forceinline__ float inf_to_nan(float f) { return is_inf(f) ? __uint_as_float(0x7FFFFFFFu) : f; }

// |f| of a finite value, 0 for an infinity (fmaxf already passes over NaN).
__device__ __forceinline__ float finite_abs(float f) { return is_inf(f) ? 0.f : fabsf(f); }

__device__ __forceinline__ void unpack8(const uint4 q, float (&f)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Two fp32 in a register pair, and their products: one instruction for both.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void f32x2_parts(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The largest of three magnitudes; NaN is passed over.
__device__ __forceinline__ float max3_abs(float a, float b, float c)
{
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight bf16 -> fp32 pairs.
__device__ __forceinline__ void unpack8_pairs(const uint4 q, uint64_t (&f)[4])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// Two pairs -> four e4m3 codes.
__device__ __forceinline__ uint32_t pack_e4m3x4(uint64_t a, uint64_t b)
{
    float f[4];
    f32x2_parts(a, f[0], f[1]);
    f32x2_parts(b, f[2], f[3]);
    return pack_e4m3x4(f[0], f[1], f[2], f[3]);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Elements c .. c+7 of a bf16 row of C elements as floats; those past the end
// read as zero.  `vec`: the row is 16-byte aligned, so whole groups load at once.
__device__ __forceinline__ uint4 load8_bf16(const uint16_t *row, int32_t c, int32_t C, bool vec)
{
    if (vec && c + 8 <= C)
        return *reinterpret_cast<const uint4 *>(row + c);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < C)
            w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements c .. c+7 of a bf16 row of C elements, from the 32 bytes that start at
// the 16-byte group its first byte lies in, `mis` bytes (even) before it; elements
// past the end are zero.
__device__ __forceinline__ uint4 shift8(uint32_t (&w)[8], uint32_t mis, int32_t c, int32_t C)
{
    // shift right by mis bytes: two words, one word, half a word
#pragma unroll
    for (int k = 0; k < 6; ++k)
        w[k] = mis & 8u ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k)
        w[k] = mis & 4u ? w[k + 1] : w[k];
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        o[k] = __funnelshift_r(w[k], w[k + 1], (mis & 2u) * 8u);
        if (c + 2 * k + 1 >= C)
            o[k] = c + 2 * k < C ? o[k] & 0xFFFFu : 0u;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight whole elements at a 2-byte aligned address: the words they lie in, shifted.
// Only words that hold one of them are read.
__device__ __forceinline__ uint4 load8_bf16_words(const uint16_t *at)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(at);
    const uint32_t *const w = reinterpret_cast<const uint32_t *>(a & ~(uintptr_t)3);
    const bool half = (a & 2u) != 0u;
    const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3], w4 = half ? w[4] : 0u;
    const uint32_t by = half ? 16u : 0u;
    return make_uint4(__funnelshift_r(w0, w1, by), __funnelshift_r(w1, w2, by), __funnelshift_r(w2, w3, by),
                      __funnelshift_r(w3, w4, by));
}

// The same from a row that is only 2-byte aligned: the 16 lanes of a half-warp
// (all of them call this) hold the vectors of 128 consecutive columns, lane l
// columns c = c0 + 8 l.  Each loads the aligned 16 bytes its vector starts in and
// takes the rest from its neighbour.  Only 16-byte granules that hold a byte of
// the row are read.
__device__ __forceinline__ uint4 load8_bf16_shifted(const uint16_t *row, int32_t c, int32_t C, bool live)
{
    const int l = (int)(threadIdx.x & 15u);
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    const uintptr_t end = reinterpret_cast<uintptr_t>(row + C);
    const uint32_t mis = (uint32_t)(at & 15u);
    const uintptr_t granule = at - mis;
    uint32_t w[8];
    uint4 q = make_uint4(0u, 0u, 0u, 0u), x = q;
    if (live && granule < end)
        q = *reinterpret_cast<const uint4 *>(granule);
    if (live && l == 15 && mis != 0u && granule + 16 < end)
        x = *reinterpret_cast<const uint4 *>(granule + 16);
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    const uint32_t extra[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t n = __shfl_down_sync(0xFFFFFFFFu, w[k], 1, 16);
        w[4 + k] = l == 15 ? extra[k] : n;
    }
    return shift8(w, mis, c, C);
}

__device__ __forceinline__ void load8_float(const float *row, int32_t c, int32_t C, bool vec, float (&f)[8])
{
    if (vec && c + 8 <= C) {
        const float4 a = *reinterpret_cast<const float4 *>(row + c);
        const float4 b = *reinterpret_cast<const float4 *>(row + c + 4);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = c + i < C ? row[c + i] : 0.f;
}

__device__ __forceinline__ void store8_bf16(uint16_t *row, int32_t c, int32_t C, bool vec, uint4 q)
{
    if (vec && c + 8 <= C) {
        *reinterpret_cast<uint4 *>(row + c) = q;
        return;
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < C)
            row[c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// The same to a row that is only 2-byte aligned, by the 16 lanes of a half-warp
// (all of them call this): each lane stores the aligned 16 bytes its vector starts
// in, with its neighbour's last elements before its own; the half-warp's first
// and last bytes, and the row's end, go element by element.  Nothing outside
// columns c .. C - 1 of the half-warp is written.
__device__ __forceinline__ void store8_bf16_shifted(uint16_t *row, int32_t c, int32_t C, bool live, uint4 q)
{
    const int l = (int)(threadIdx.x & 15u);
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    const uint32_t mis = (uint32_t)(at & 15u);
    uint32_t w[8];  // the neighbour's vector, then this one
    w[4] = q.x, w[5] = q.y, w[6] = q.z, w[7] = q.w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = __shfl_up_sync(0xFFFFFFFFu, w[4 + k], 1, 16);
    if (!live)
        return;
    const int32_t end = c + 8 < C ? 8 : C - c;  // this vector's live elements
    if ((l > 0 || mis == 0u) && C - c >= 8 - (int32_t)(mis >> 1)) {
        // bytes 16 - mis .. 31 - mis of the two vectors: shift right by 16 - mis
        const uint32_t by = 16u - mis;
        uint32_t s[5];
#pragma unroll
        for (int k = 0; k < 5; ++k)  // by / 4 words: 1 to 4
            s[k] = by >= 16u ? (k < 4 ? w[k + 4] : 0u)
                             : (by >= 12u ? w[k + 3] : (by >= 8u ? w[k + 2] : (by >= 4u ? w[k + 1] : w[k])));
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = __funnelshift_r(s[k], s[k + 1], (by & 2u) * 8u);
        *reinterpret_cast<uint4 *>(at - mis) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        // this vector's part of its first granule (and, for later lanes, the
        // neighbour's part of it)
        const int32_t own = 8 - (int32_t)(mis >> 1);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < own && j < end)
                row[c + j] = (uint16_t)(w[4 + (j >> 1)] >> (16 * (j & 1)));
        if (l > 0) {
#pragma unroll
            for (int j = 1; j < 8; ++j)
                if (j >= own)
                    row[c - 8 + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
    // what no later lane stores: the last lane's rest, or that of the row's last vector
    if (l == 15 || c + 8 >= C) {
        const int32_t own = 8 - (int32_t)(mis >> 1);
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (j >= own && j < end)
                row[c + j] = (uint16_t)(w[4 + (j >> 1)] >> (16 * (j & 1)));
    }
}

// Codes c .. c+7 of a row (rows are 16-byte aligned).
__device__ __forceinline__ void store8_codes(uint8_t *row, int32_t c, int32_t C, uint2 q)
{
    if (c + 8 <= C) {
        *reinterpret_cast<uint2 *>(row + c) = q;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < C)
            row[c + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

}  // namespace wstma
