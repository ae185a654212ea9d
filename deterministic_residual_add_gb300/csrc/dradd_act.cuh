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

// act(z).  The tails of both forms of gelu are computed as z times a small
// number, not as a difference of numbers near 1.
template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == DRADD_ACT_RELU)
        return z < 0.0f ? 0.0f : z;
    else if constexpr (ACT == DRADD_ACT_GELU)
        return 0.5f * z * erfcf(z * -0.70710678118654752f);
    else if constexpr (ACT == DRADD_ACT_GELU_TANH)
        return z * logistic(2.0f * kGeluC * fmaf(kGeluA * z * z, z, z));
    else if constexpr (ACT == DRADD_ACT_SILU)
        return z * logistic(z);
    else
        return z;
}

// act'(z); where its first factor has vanished, z times it counts as 0
// however large z is.
template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == DRADD_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == DRADD_ACT_GELU) {
        const float g = 0.3989422804014327f * exp2_fast(-0.5f * kLog2e * z * z);  // the normal density
        const float f = 0.5f * erfcf(z * -0.70710678118654752f);
        return g == 0.0f ? f : fmaf(z, g, f);
    } else if constexpr (ACT == DRADD_ACT_GELU_TANH) {
        const float f = logistic(2.0f * kGeluC * fmaf(kGeluA * z * z, z, z));
        const float w = f * (1.0f - f);
        return w == 0.0f ? f : fmaf(z * w, 2.0f * kGeluC * fmaf(3.0f * kGeluA * z, z, 1.0f), f);
    } else if constexpr (ACT == DRADD_ACT_SILU) {
        const float f = logistic(z), w = f * (1.0f - f);
        return w == 0.0f ? f : fmaf(z, w, f);
    } else {
        return 1.0f;
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

// z = act'(z).
template <int N>
__device__ __forceinline__ void act_slopes(float (&z)[N], int act)
{
    switch (act) {
    case DRADD_ACT_RELU: act_slopes<DRADD_ACT_RELU>(z); break;
    case DRADD_ACT_GELU: act_slopes<DRADD_ACT_GELU>(z); break;
    case DRADD_ACT_GELU_TANH: act_slopes<DRADD_ACT_GELU_TANH>(z); break;
    case DRADD_ACT_SILU: act_slopes<DRADD_ACT_SILU>(z); break;
    default: act_slopes<DRADD_ACT_NONE>(z); break;
    }
}

}  // namespace dradd
