// Activations of the feed-forward operators and their slopes, in fp32, and the
// 8-bit values of a checkpoint.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ffn_kernels.h"
#include "fp8_format.cuh"

namespace wstma {

// 1 / (1 + exp(-x)).  exp's overflow ends at 0, as it should.
__device__ __forceinline__ float ffn_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// a (x + 0.044715 x^3) with a = 2 sqrt(2 / pi): gelu by tanh is x sigmoid of it, since
// (1 + tanh(y)) / 2 = sigmoid(2 y).  No cancellation for either sign.
__device__ __forceinline__ float ffn_tanh_arg(float x)
{
    return 1.5957691216057308f * fmaf(0.044715f * x * x, x, x);
}

// Phi(x), the normal distribution's, and e = exp(-x^2 / 2).  The lower tail is e times a
// function of |x| that decays like 1 / |x|: a polynomial in u = 1 / (1 + q |x|), fitted to it by
// least squares whose weights were raised where the relative error was largest, over |x| <= 13.4.
// Off by 4.4e-7 of Phi at most, in the tail too, where 1 + erf cancels; and the slope needs e
// besides.  With erfcf the slope kernel was bound by its arithmetic (6143 x 5999: 115 us, of which
// HBM's are 33).
__device__ __forceinline__ void ffn_normal(float x, float &cdf, float &e)
{
    const float u = __fdividef(1.0f, fmaf(0.304055929f, fabsf(x), 1.0f));
    e = __expf(-0.5f * x * x);
    float t = 0.0368540585f;
    t = fmaf(t, u, -0.155187115f);
    t = fmaf(t, u, 0.191853642f);
    t = fmaf(t, u, -0.0428636521f);
    t = fmaf(t, u, 0.123422652f);
    t = fmaf(t, u, 0.102475412f);
    t = fmaf(t, u, 0.122187749f);
    t = fmaf(t, u, 0.121257305f);
    t *= u * e;
    cdf = x < 0.0f ? t : 1.0f - t;
}

template <int A>
__device__ __forceinline__ float ffn_act(float x)
{
    if constexpr (A == kActRelu)
        return x > 0.0f || x != x ? x : 0.0f;
    if constexpr (A == kActSilu)
        return x * ffn_sigmoid(x);
    if constexpr (A == kActGelu) {
        float c, e;
        ffn_normal(x, c, e);
        return x * c;
    }
    if constexpr (A == kActGeluTanh)
        return x * ffn_sigmoid(ffn_tanh_arg(x));
    return x;
}

// act(x) and act'(x).
template <int A>
__device__ __forceinline__ void ffn_act_slope(float x, float &a, float &d)
{
    if constexpr (A == kActRelu) {
        a = x > 0.0f || x != x ? x : 0.0f;
        d = x > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (A == kActSilu) {
        const float s = ffn_sigmoid(x);
        a = x * s;
        d = fmaf(a, 1.0f - s, s);
    } else if constexpr (A == kActGelu) {
        float c, e;
        ffn_normal(x, c, e);
        a = x * c;
        d = fmaf(0.39894228040143268f * x, e, c);
    } else if constexpr (A == kActGeluTanh) {
        const float s = ffn_sigmoid(ffn_tanh_arg(x));
        a = x * s;
        // beyond 30 the slope of the sigmoid is 0, and x^2 times it must not become inf * 0
        const float y = fminf(fmaxf(x, -30.0f), 30.0f);
        d = fmaf(y * s * (1.0f - s), 1.5957691216057308f * fmaf(3.0f * 0.044715f * y, y, 1.0f), s);
    } else {
        a = x;
        d = 1.0f;
    }
}

// f(std::integral_constant) for the activation `act`: the choice is made once, outside f's loops.
template <int A>
struct FfnActTag {
    static constexpr int value = A;
};

template <typename F>
__device__ __forceinline__ void ffn_with_act(int32_t act, F f)
{
    switch (act) {
    case kActRelu: f(FfnActTag<kActRelu>{}); break;
    case kActSilu: f(FfnActTag<kActSilu>{}); break;
    case kActGelu: f(FfnActTag<kActGelu>{}); break;
    case kActGeluTanh: f(FfnActTag<kActGeluTanh>{}); break;
    default: f(FfnActTag<kActNone>{}); break;
    }
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 2^(byte - 127), of an e8m0 byte; 255 stands for NaN.
__device__ __forceinline__ float ffn_scale(uint32_t byte)
{
    return byte == 0u ? __uint_as_float(0x00400000u) : byte == 255u ? __uint_as_float(0x7FFFFFFFu)
                                                                     : __uint_as_float(byte << 23);
}

// Two e4m3 codes (the low 16 bits of `codes`) as fp32.
__device__ __forceinline__ void ffn_from_e4m3x2(uint32_t codes, float &lo, float &hi)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    lo = f.x;
    hi = f.y;
}

}  // namespace wstma
