// Activations of the dense layer and their slopes, in fp32.
#pragma once

#include <cstdint>

#include "pairs.cuh"

namespace mxfp4 {

// The ABI's MXFP4_ACT_* codes.
enum class Act { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ F2 rcp2(F2 a)
{
    const float2 p = parts(a);
    return f2(rcp_approx(p.x), rcp_approx(p.y));
}
__device__ __forceinline__ F2 ex2_2(F2 a)
{
    const float2 p = parts(a);
    return f2(ex2_approx(p.x), ex2_approx(p.y));
}

// sigmoid(u) = 1 / (1 + exp(-u)); 0 where exp(-u) passes the largest number.
// u log2(e) is given.
__device__ __forceinline__ F2 sigmoid2(F2 u_log2e) { return rcp2(f2(1.0f) + ex2_2(f2(-1.0f) * u_log2e)); }

// The normal distribution: phi(z) = exp(-z^2 / 2) / sqrt(2 pi) and Phi(z).
// With x = |z|, Phi(-x) exp(x^2 / 2) is smooth and falls like 1 / x, so it is
// t P(t) with t = 1 / (1 + 3/8 x) and a polynomial P of degree 8, fitted to that
// function's values on t in (0, 1] for the smallest largest relative error
// (2.2e-7; 5.1e-7 with P's own rounding).  The lower tail comes out of it to that relative
// precision, without a subtraction, and both phi and Phi from one exponential and
// one reciprocal.
__device__ __forceinline__ F2 normal_tail2(F2 minus_abs, F2 e)
{
    const F2 t = rcp2(fma2(f2(-0.375f), minus_abs, f2(1.0f)));
    F2 p = f2(-0.032911055f);
    p = fma2(p, t, f2(0.136879951f));
    p = fma2(p, t, f2(-0.186521217f));
    p = fma2(p, t, f2(0.0506323874f));
    p = fma2(p, t, f2(0.0156279318f));
    p = fma2(p, t, f2(0.0886382312f));
    p = fma2(p, t, f2(0.12844570f));
    p = fma2(p, t, f2(0.149604589f));
    p = fma2(p, t, f2(0.149603382f));
    return e * (t * p);
}

// exp(-z^2 / 2)
__device__ __forceinline__ F2 bell2(F2 z) { return ex2_2(f2(-0.72134752f) * (z * z)); }

__device__ __forceinline__ void normal2(F2 z, F2 &below, F2 &density)
{
    const float2 zs = parts(z);
    const F2 e = bell2(z), tail = normal_tail2(f2(-fabsf(zs.x), -fabsf(zs.y)), e);
    const float2 low = parts(tail), high = parts(fma2(tail, f2(-1.0f), f2(1.0f)));
    below = f2(zs.x < 0.0f ? low.x : high.x, zs.y < 0.0f ? low.y : high.y);
    density = f2(0.39894228f) * e;
}

// act(z) and act'(z) of two values.  GELU's tanh form is z sigmoid(2 u), u = sqrt(2 / pi)
// (z + 0.044715 z^3), as (1 + tanh u) / 2 = sigmoid(2 u).  NaN stays NaN in act(z).
template <Act A>
__device__ __forceinline__ void act_and_slope2(F2 z, F2 &h, F2 &slope)
{
    if constexpr (A == Act::kRelu) {
        const float2 p = parts(z);
        h = f2(p.x < 0.0f ? 0.0f : p.x, p.y < 0.0f ? 0.0f : p.y);
        slope = f2(p.x <= 0.0f ? 0.0f : 1.0f, p.y <= 0.0f ? 0.0f : 1.0f);
    } else if constexpr (A == Act::kGelu) {
        F2 below, density;
        normal2(z, below, density);
        h = z * below;
        slope = fma2(z, density, below);
    } else if constexpr (A == Act::kGeluTanh) {
        // 2 u log2(e) = z (2.302208 + 0.10294324 z^2)
        const F2 zz = z * z;
        const F2 g = sigmoid2(z * fma2(f2(0.10294324f), zz, f2(2.3022082f)));
        h = z * g;
        // The slope's factor stays finite where z^2 does not: h (1 - g) is 0 long before, and 0 times infinity is NaN.
        const float2 p = parts(zz);
        slope = fma2(h * fma2(g, f2(-1.0f), f2(1.0f)), fma2(f2(0.214064449f), f2(fminf(p.x, 1e30f), fminf(p.y, 1e30f)), f2(1.59576912f)), g);
    } else if constexpr (A == Act::kSilu) {
        const F2 g = sigmoid2(f2(1.44269504f) * z);
        h = z * g;
        slope = fma2(h, fma2(g, f2(-1.0f), f2(1.0f)), g);
    } else {
        h = z;
        slope = f2(1.0f);
    }
}

template <Act A>
__device__ __forceinline__ F2 act_value2(F2 z)
{
    if constexpr (A == Act::kGelu) {
        // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
        const float2 p = parts(z);
        // (bounded, as Phi is 0 long before and infinity times 0 is NaN; a NaN comes through `above`)
        const F2 minus = f2(fmaxf(-fabsf(p.x), -1e30f), fmaxf(-fabsf(p.y), -1e30f)),
                 above = f2(p.x < 0.0f ? 0.0f : p.x, p.y < 0.0f ? 0.0f : p.y);
        return fma2(minus, normal_tail2(minus, bell2(z)), above);
    }
    F2 h, slope;
    act_and_slope2<A>(z, h, slope);
    return h;
}

// Calls f(std::integral_constant-like tag) for the runtime code of an activation.
template <Act A>
struct ActTag {
    static constexpr Act value = A;
};
template <typename F>
inline auto with_act(int act, F f)
{
    switch (act) {
    case 1: return f(ActTag<Act::kRelu>{});
    case 2: return f(ActTag<Act::kGelu>{});
    case 3: return f(ActTag<Act::kGeluTanh>{});
    case 4: return f(ActTag<Act::kSilu>{});
    default: return f(ActTag<Act::kNone>{});
    }
}

}  // namespace mxfp4
