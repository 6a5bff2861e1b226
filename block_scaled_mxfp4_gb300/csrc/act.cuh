// Activations of the dense layer and their slopes, in fp32.
#pragma once

#include <cstdint>

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

// sigmoid(u) = 1 / (1 + exp(-u)); 0 where exp(-u) passes the largest number.
__device__ __forceinline__ float sigmoid_approx(float u) { return rcp_approx(1.0f + ex2_approx(-1.44269504f * u)); }

// The normal distribution: phi(z) = exp(-z^2 / 2) / sqrt(2 pi) and Phi(z).
// With x = |z|, Phi(-x) exp(x^2 / 2) is smooth and falls like 1 / x, so it is
// t P(t) with t = 1 / (1 + 3/8 x) and a polynomial P of degree 8, fitted to that
// function's values on t in (0, 1] for the smallest largest relative error
// (2.2e-7; 5.1e-7 with P's own rounding).  The lower tail comes out of it to that relative
// precision, without a subtraction, and both phi and Phi from one exponential and
// one reciprocal.
__device__ __forceinline__ void normal_approx(float z, float &below, float &density)
{
    const float x = fabsf(z);
    const float t = rcp_approx(fmaf(0.375f, x, 1.0f));
    const float e = ex2_approx(-0.72134752f * z * z);
    float p = -0.032911055f;
    p = fmaf(p, t, 0.136879951f);
    p = fmaf(p, t, -0.186521217f);
    p = fmaf(p, t, 0.0506323874f);
    p = fmaf(p, t, 0.0156279318f);
    p = fmaf(p, t, 0.0886382312f);
    p = fmaf(p, t, 0.12844570f);
    p = fmaf(p, t, 0.149604589f);
    p = fmaf(p, t, 0.149603382f);
    const float tail = e * (t * p);
    below = z < 0.0f ? tail : 1.0f - tail;
    density = 0.39894228f * e;
}

// act(z).  GELU's tanh form is z sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3),
// as (1 + tanh u) / 2 = sigmoid(2 u).  NaN stays NaN.
template <Act A>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (A == Act::kRelu) {
        return z < 0.0f ? 0.0f : z;
    } else if constexpr (A == Act::kGelu) {
        float below, density;
        normal_approx(z, below, density);
        return z * below;
    } else if constexpr (A == Act::kGeluTanh) {
        return z * sigmoid_approx(z * fmaf(0.0713548163f, z * z, 1.59576912f));
    } else if constexpr (A == Act::kSilu) {
        return z * sigmoid_approx(z);
    } else {
        return z;
    }
}

// act(z) and act'(z).
template <Act A>
__device__ __forceinline__ void act_and_slope(float z, float &h, float &slope)
{
    if constexpr (A == Act::kRelu) {
        h = z < 0.0f ? 0.0f : z;
        slope = z <= 0.0f ? 0.0f : 1.0f;
    } else if constexpr (A == Act::kGelu) {
        float below, density;
        normal_approx(z, below, density);
        h = z * below;
        slope = fmaf(z, density, below);
    } else if constexpr (A == Act::kGeluTanh) {
        const float g = sigmoid_approx(z * fmaf(0.0713548163f, z * z, 1.59576912f));
        h = z * g;
        slope = fmaf(h * (1.0f - g), fmaf(0.214064449f, z * z, 1.59576912f), g);
    } else if constexpr (A == Act::kSilu) {
        const float g = sigmoid_approx(z);
        h = z * g;
        slope = fmaf(h, 1.0f - g, g);
    } else {
        h = z;
        slope = 1.0f;
    }
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
