// Activations of the feed-forward operators and their slopes, in fp32, and the
// 8-bit values of a checkpoint.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ffn_kernels.h"
#include "fp8_format.cuh"

namespace wstma {

// 2^x and 1 / x by the special-function unit alone, with subnormal results at 0: the forms that keep
// subnormals take three to four instructions more, and nothing here needs those.
__device__ __forceinline__ float ffn_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float ffn_reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// Two values side by side, one instruction for both (Blackwell's packed fp32 arithmetic): the epilogues
// that take slopes are bound by the instructions they issue.
struct Pair {
    uint64_t v;
};

__device__ __forceinline__ Pair pair(float lo, float hi) { return {f32x2(lo, hi)}; }
__device__ __forceinline__ Pair both(float x) { return {f32x2(x, x)}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) { return {mul_f32x2(a.v, b.v)}; }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) { return {fma_f32x2(a.v, b.v, c.v)}; }
__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// f of each half
template <typename F>
__device__ __forceinline__ Pair each(Pair a, F f)
{
    float lo, hi;
    f32x2_parts(a.v, lo, hi);
    return pair(f(lo), f(hi));
}

__device__ __forceinline__ uint32_t bf16_pair(Pair a)
{
    float lo, hi;
    f32x2_parts(a.v, lo, hi);
    return bf16_pair(lo, hi);
}

// 1 / (1 + exp(-x)).  exp's overflow ends at 0, as it should.
__device__ __forceinline__ Pair ffn_sigmoid(Pair x)
{
    const Pair e = each(x * both(-kLog2e), [](float v) { return ffn_exp2(v); });
    return each(e + both(1.0f), [](float v) { return ffn_reciprocal(v); });
}

// Phi(x), the normal distribution's, and e = exp(-x^2 / 2).  The lower tail is e times a
// function of |x| that decays like 1 / |x|: a polynomial in u = 1 / (1 + q |x|), fitted to it by
// least squares whose weights were raised where the relative error was largest, over |x| <= 13.4, to 1.0e-7.
// In 32 bits, exp2's own error aside, off by 4.5e-7 of Phi at most down to x = -2, where 1 + erf cancels, 7.6e-7 to -4, 2.7e-6 to
// -8 and 5e-6 to -10: x^2 is rounded before it is an exponent, which a result in bf16 does not show and one in
// fp32 does.  The slope needs e besides.  With erfcf the slope kernel was bound by its arithmetic (6143 x 5999: 115 us, of which
// HBM's are 33).
__device__ __forceinline__ void ffn_normal(Pair x, Pair &cdf, Pair &e)
{
    const Pair u = each(x, [](float v) { return ffn_reciprocal(fmaf(0.304055929f, fabsf(v), 1.0f)); });
    e = each(x * x * both(-0.5f * kLog2e), [](float v) { return ffn_exp2(v); });
    Pair t = fma2(both(0.0368540585f), u, both(-0.155187115f));
    t = fma2(t, u, both(0.191853642f));
    t = fma2(t, u, both(-0.0428636521f));
    t = fma2(t, u, both(0.123422652f));
    t = fma2(t, u, both(0.102475412f));
    t = fma2(t, u, both(0.122187749f));
    t = fma2(t, u, both(0.121257305f));
    t = t * (u * e);
    float x0, x1, t0, t1;
    f32x2_parts(x.v, x0, x1);
    f32x2_parts(t.v, t0, t1);
    cdf = pair(x0 < 0.0f ? t0 : 1.0f - t0, x1 < 0.0f ? t1 : 1.0f - t1);
}

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// act(x) and act'(x); gelu by tanh is x sigmoid(2 sqrt(2 / pi) (x + 0.044715 x^3)), since
// (1 + tanh(y)) / 2 = sigmoid(2 y): no cancellation for either sign.
template <int A>
__device__ __forceinline__ void ffn_act_slope(Pair x, Pair &a, Pair &d)
{
    if constexpr (A == kActRelu) {
        a = each(x, [](float v) { return v > 0.0f || v != v ? v : 0.0f; });
        d = each(x, [](float v) { return v > 0.0f ? 1.0f : 0.0f; });
    } else if constexpr (A == kActSilu) {
        const Pair s = ffn_sigmoid(x);
        a = x * s;
        d = fma2(a, fma2(s, both(-1.0f), both(1.0f)), s);
    } else if constexpr (A == kActGelu) {
        Pair c, e;
        ffn_normal(x, c, e);
        a = x * c;
        d = fma2(both(0.39894228040143268f) * x, e, c);
    } else if constexpr (A == kActGeluTanh) {
        const Pair s = ffn_sigmoid(x * fma2(x * x, both(kTanhScale * 0.044715f), both(kTanhScale)));
        a = x * s;
        // beyond 30 the slope of the sigmoid is 0, and x^2 times it must not become inf * 0
        const Pair y = each(x, [](float v) { return fminf(fmaxf(v, -30.0f), 30.0f); });
        const Pair rise = y * s * fma2(s, both(-1.0f), both(1.0f));
        d = fma2(rise, fma2(y * y, both(kTanhScale * 3.0f * 0.044715f), both(kTanhScale)), s);
    } else {
        a = x;
        d = both(1.0f);
    }
}

template <int A>
__device__ __forceinline__ Pair ffn_act(Pair x)
{
    Pair a, d;
    ffn_act_slope<A>(x, a, d);  // the slope is not computed where it is not used
    return a;
}

template <int A>
__device__ __forceinline__ float ffn_act(float x)
{
    float lo, hi;
    f32x2_parts(ffn_act<A>(pair(x, x)).v, lo, hi);
    return lo;
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

// Two bf16, or two e4m3 codes (the low 16 bits of `codes`), as fp32.
__device__ __forceinline__ Pair pair_of_bf16(uint32_t w) { return pair(bf16_low(w), bf16_high(w)); }

__device__ __forceinline__ Pair pair_of_e4m3(uint32_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pair(f.x, f.y);
}

}  // namespace wstma
