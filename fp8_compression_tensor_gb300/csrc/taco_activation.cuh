// taco_activation.cuh -- the activations of the training operators and their
// slopes, two values at a time: GELU (both forms) and SiLU.
#pragma once

#include <cfloat>

#include "taco_train.cuh"

namespace taco {
namespace {

constexpr float kTanhA = 0.7978845608028654f, kTanhB = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f, kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float reciprocal_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// |v|, for positive v at most 30, and a NaN kept.  In the gradient the bound keeps +infinity from meeting the tail's
// zero; -infinity does meet it, as in u Phi(u) = -infinity 0, and comes out as NaN.
__device__ __forceinline__ float bounded_abs(float v)
{
    float r;
    asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(v), "f"(30.f), "f"(-v));
    return r;
}

// Upper tail q = 1 - Phi(a) of the normal distribution for a = |u|, and
// E = exp(-a^2 / 2), which the exponential flushes to zero below 2^-126 (a above
// 13.2).  q = erfc(a / sqrt 2) / 2 equals E t Q(t), t = 1 / (1 + 0.3 a): erfc(z)
// exp(z^2) is smooth and falls like 1/z, so a polynomial in t follows it on the
// whole half line.  Q (degree 7) is a least-squares fit reweighted towards the
// smallest largest relative error on 0 <= a <= 14, 1.7e-7 with the coefficients as
// written.  In binary32 the tail is off by at most 2.5e-7 in absolute terms; its
// relative error grows with the exponent's rounding, which weighs a^2 / 2: measured
// 7e-7 up to a = 4, 3.3e-6 up to 9, 7e-6 up to 13.  One exponential and one
// reciprocal serve Phi and, in the gradient, the density too.
//   gelu(u)  = u Phi(u) = u q for u < 0 and u (1 - q) otherwise, which is max(u, 0) - a q
//   gelu'(u) = Phi(u) + u phi(u) = r for u < 0 and 1 - r otherwise, r = q - a phi(a)
// The value alone takes the first form: 8192 x 16384 bf16 with records 132 us against 134.  The gradient takes the
// second one, whose bounded a it has.
__device__ __forceinline__ float2 normal_tail2(float2 a, float2 &e)
{
    const float2 x = mul2(mul2(a, a), both(-0.5f * kLog2e));
    e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
    const float2 d = fma2(a, both(0.3f), both(1.f));
    const float2 t = make_float2(reciprocal_fast(d.x), reciprocal_fast(d.y));
    float2 q = both(0.03567478060722351f);
    q = fma2(q, t, both(-0.1572030931711197f));
    q = fma2(q, t, both(0.20635348558425903f));
    q = fma2(q, t, both(-0.05368363484740257f));
    q = fma2(q, t, both(0.1285616159439087f));
    q = fma2(q, t, both(0.09991350024938583f));
    q = fma2(q, t, both(0.12075395882129669f));
    q = fma2(q, t, both(0.11962930113077164f));
    return mul2(mul2(q, t), e);
}

// 1 / (1 + exp(-2 v)) = (1 + tanh v) / 2 for v = a (u + b u^3).
__device__ __forceinline__ float2 tanh_gate2(float2 u)
{
    const float2 poly = fma2(mul2(u, u), both(kTanhA * kTanhB), both(kTanhA));
    const float2 x = mul2(mul2(poly, u), both(-2.f * kLog2e));
    return make_float2(reciprocal_fast(1.f + exp2_fast(x.x)), reciprocal_fast(1.f + exp2_fast(x.y)));
}

template <bool TANH>
__device__ __forceinline__ float2 gelu_value2(float2 u)
{
    if (TANH)
        return mul2(u, tanh_gate2(u));
    float2 e;
    const float2 q = normal_tail2(make_float2(fabsf(u.x), fabsf(u.y)), e), p = add2(both(1.f), make_float2(-q.x, -q.y));
    return mul2(u, make_float2(u.x < 0.f ? q.x : p.x, u.y < 0.f ? q.y : p.y));
}

// gelu(u) and its slope.
template <bool TANH>
__device__ __forceinline__ void gelu_both2(float2 u, float2 &y, float2 &slope)
{
    if (TANH) {
        const float2 g = tanh_gate2(u);
        // Beyond |u| = 16 the gate is 0 or 1 and its slope 0; the clamp keeps u^2 finite.
        const float2 c = make_float2(fminf(fmaxf(u.x, -16.f), 16.f), fminf(fmaxf(u.y, -16.f), 16.f));
        const float2 inner = fma2(mul2(c, c), both(6.f * kTanhA * kTanhB), both(2.f * kTanhA));
        const float2 rest = fma2(g, make_float2(-g.x, -g.y), g);          // g (1 - g)
        slope = fma2(mul2(c, inner), rest, g);
        // What is not above -infinity gives NaN, as y = u g does; it does not pass the clamp.  Asked of u: asked of y, 8192 x
        // 16384 takes 169 us against 160.
        if (!(u.x >= -FLT_MAX))
            slope.x = __uint_as_float(0x7fc00000u);
        if (!(u.y >= -FLT_MAX))
            slope.y = __uint_as_float(0x7fc00000u);
        y = mul2(u, g);
    } else {
        float2 e;
        const float2 a = make_float2(bounded_abs(u.x), bounded_abs(u.y)), minus = make_float2(-a.x, -a.y);
        const float2 q = normal_tail2(a, e);
        const float2 r = fma2(mul2(minus, both(kInvSqrt2Pi)), e, q);
        // A choice rather than 1/2 + sign(u) (1/2 - r), in which r below 0 would lose what lies under 3e-8.
        const float2 h = add2(both(1.f), make_float2(-r.x, -r.y));
        slope = make_float2(u.x < 0.f ? r.x : h.x, u.y < 0.f ? r.y : h.y);
        y = fma2(minus, q, make_float2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
    }
}

// silu(g) = g p with p = 1 / (1 + exp(-g)), and its slope p (1 + g (1 - p)).  The
// exponential's error grows with the rounding of g log2(e), to 1e-6 of p at g =
// -16; above, 1 / (1 + e) damps it.  Below g = -87.3 p is flushed to zero, and g p,
// smaller than 2^-119 there, with it.  g bounded by 80 in the slope keeps +infinity
// from meeting 1 - p = 0 (slope 1); -infinity meets p = 0 in both (NaN).
__device__ __forceinline__ float2 silu_gate2(float2 g)
{
    const float2 x = mul2(g, both(-kLog2e));
    const float2 d = add2(make_float2(exp2_fast(x.x), exp2_fast(x.y)), both(1.f));
    return make_float2(reciprocal_fast(d.x), reciprocal_fast(d.y));
}

// Activations (taco_activation_t).
constexpr int kSilu = 0, kGelu = 1, kGeluTanh = 2;

template <int ACT>
__device__ __forceinline__ float2 activation2(float2 g)
{
    return ACT == kSilu ? mul2(g, silu_gate2(g)) : gelu_value2<ACT == kGeluTanh>(g);
}

// The activation and its slope.
template <int ACT>
__device__ __forceinline__ void activation_both2(float2 g, float2 &y, float2 &slope)
{
    if (ACT != kSilu) {
        gelu_both2<ACT == kGeluTanh>(g, y, slope);
        return;
    }
    const float2 p = silu_gate2(g), c = make_float2(fminf(g.x, 80.f), fminf(g.y, 80.f));
    const float2 q = add2(both(1.f), make_float2(-p.x, -p.y));
    slope = mul2(p, fma2(c, q, both(1.f)));
    y = mul2(g, p);
}

}  // namespace
}  // namespace taco
