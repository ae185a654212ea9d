// dradd_act.cuh -- activations of dradd_linear.h and their derivatives, fp32.
#pragma once

#include <cstdint>

#include "dradd_linear.h"

namespace dradd {

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 1 / (1 + e^-x).  The two approximations are off by 2^-22 each, the
// exponent by |x| 2^-23: at most 2^-16 of the result (|x| < 88, behind which
// it is 0 or 1), an eighth of fp16's half step.
__device__ __forceinline__ float logistic(float x) { return rcp_fast(1.0f + exp2_fast(-kLog2e * x)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// erfc(x) for x >= 0 as e^(-x^2) times this: t e^(P(t)), t = 1 / (1 + x / 2),
// with the Chebyshev fit of Press, Flannery, Teukolsky and Vetterling
// ("Numerical Recipes", erfcc), whose relative error is below 1.2e-7
// everywhere.  erfcf took 10.6 us for a tile's 32768 values.
__device__ __forceinline__ float erfc_factor(float x)
{
    const float t = rcp_fast(fmaf(0.5f, x, 1.0f));
    float p = 0.17087277f;
    p = fmaf(p, t, -0.82215223f);
    p = fmaf(p, t, 1.48851587f);
    p = fmaf(p, t, -1.13520398f);
    p = fmaf(p, t, 0.27886807f);
    p = fmaf(p, t, -0.18628806f);
    p = fmaf(p, t, 0.09678418f);
    p = fmaf(p, t, 0.37409196f);
    p = fmaf(p, t, 1.00002368f);
    p = fmaf(p, t, -1.26551223f);
    return t * exp2_fast(kLog2e * p);
}

// Phi(z), the normal distribution's function, and e^(-z^2 / 2).  The tail on
// the left is a small number of its own, not a difference of numbers near 1.
__device__ __forceinline__ float normal_cdf(float z, float& e)
{
    const float x = fabsf(z) * 0.70710678118654752f;
    e = exp2_fast(-kLog2e * (x * x));
    const float tail = 0.5f * e * erfc_factor(x);
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == DRADD_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;
    } else if constexpr (ACT == DRADD_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    } else if constexpr (ACT == DRADD_ACT_GELU_TANH) {
        return z * logistic(2.0f * kGeluC * fmaf(kGeluA * z * z, z, z));
    } else if constexpr (ACT == DRADD_ACT_SILU) {
        return z * logistic(z);
    } else {
        return z;
    }
}

// act'(z); where its first factor has vanished, z times it counts as 0
// however large z is.
template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == DRADD_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == DRADD_ACT_GELU) {
        float e;
        const float f = normal_cdf(z, e);
        return e == 0.0f ? f : fmaf(z * e, 0.3989422804014327f, f);
    } else if constexpr (ACT == DRADD_ACT_GELU_TANH) {
        const float f = logistic(2.0f * kGeluC * fmaf(kGeluA * z * z, z, z));
        const float w = f * (1.0f - f);
        return w == 0.0f ? f : fmaf(z * w, 2.0f * kGeluC * fmaf(3.0f * kGeluA * z, z, 1.0f), f);
    } else {
        static_assert(ACT == DRADD_ACT_SILU);
        const float f = logistic(z), w = f * (1.0f - f);
        return w == 0.0f ? f : fmaf(z, w, f);
    }
}

template <int ACT, int N>
__device__ __forceinline__ void act_values(float (&z)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        z[j] = act_value<ACT>(z[j]);
}

template <int ACT, int N>
__device__ __forceinline__ void act_slopes(float (&z)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        z[j] = act_slope<ACT>(z[j]);
}

// z = act(z), one choice for all.
template <int N>
__device__ __forceinline__ void act_values(float (&z)[N], int act)
{
    switch (act) {
    case DRADD_ACT_RELU: act_values<DRADD_ACT_RELU>(z); break;
    case DRADD_ACT_GELU: act_values<DRADD_ACT_GELU>(z); break;
    case DRADD_ACT_GELU_TANH: act_values<DRADD_ACT_GELU_TANH>(z); break;
    case DRADD_ACT_SILU: act_values<DRADD_ACT_SILU>(z); break;
    default: break;
    }
}

// z = act'(z); not for DRADD_ACT_NONE, whose dz is the gradient that comes in.
template <int N>
__device__ __forceinline__ void act_slopes(float (&z)[N], int act)
{
    switch (act) {
    case DRADD_ACT_RELU: act_slopes<DRADD_ACT_RELU>(z); break;
    case DRADD_ACT_GELU: act_slopes<DRADD_ACT_GELU>(z); break;
    case DRADD_ACT_GELU_TANH: act_slopes<DRADD_ACT_GELU_TANH>(z); break;
    default: act_slopes<DRADD_ACT_SILU>(z); break;
    }
}

}  // namespace dradd
