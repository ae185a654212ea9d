// dradd_act.cuh -- activations of dradd_linear.h and their derivatives, fp32.
#pragma once

#include <cstdint>

#include "dradd_device.cuh"
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

// Two values at a time: the pairs share their instructions (add, multiply and
// fma on two fp32 numbers at once), all but the approximations.  One by one
// the epilogue of a gradient took 15000 cycles for a tile of gelu_tanh.
struct Two {
    float a, b;
};
__device__ __forceinline__ Two both(float v) { return {v, v}; }
__device__ __forceinline__ Two operator+(Two x, Two y)
{
    Two d;
    add2_rn(x.a, x.b, y.a, y.b, d.a, d.b);
    return d;
}
__device__ __forceinline__ Two operator*(Two x, Two y)
{
    Two d;
    mul2_rn(x.a, x.b, y.a, y.b, d.a, d.b);
    return d;
}
__device__ __forceinline__ Two fma2(Two x, Two y, Two z)
{
    Two d;
    fma2_rn(x.a, x.b, y.a, y.b, z.a, z.b, d.a, d.b);
    return d;
}
__device__ __forceinline__ Two exp2_fast(Two x) { return {exp2_fast(x.a), exp2_fast(x.b)}; }
__device__ __forceinline__ Two rcp_fast(Two x) { return {rcp_fast(x.a), rcp_fast(x.b)}; }

// 1 / (1 + 2^-y), y = log2(e) x: the logistic function.  The two
// approximations are off by 2^-22 each, the exponent by |x| 2^-22: at most
// 2^-15 of the result (|x| < 88, behind which it is 0 or 1), a sixteenth of
// fp16's half step.
__device__ __forceinline__ Two logistic2(Two minus_y) { return rcp_fast(both(1.0f) + exp2_fast(minus_y)); }

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// erfc(x) for x >= 0 as e^(-x^2) times this: t e^(P(t)), t = 1 / (1 + x / 2),
// with the Chebyshev fit of Press, Flannery, Teukolsky and Vetterling
// ("Numerical Recipes", erfcc), whose relative error is below 1.2e-7
// everywhere.  erfcf took 10.6 us for a tile's 32768 values.
__device__ __forceinline__ Two erfc_factor(Two x)
{
    const Two t = rcp_fast(fma2(both(0.5f), x, both(1.0f)));
    Two p = fma2(both(0.17087277f), t, both(-0.82215223f));
    p = fma2(p, t, both(1.48851587f));
    p = fma2(p, t, both(-1.13520398f));
    p = fma2(p, t, both(0.27886807f));
    p = fma2(p, t, both(-0.18628806f));
    p = fma2(p, t, both(0.09678418f));
    p = fma2(p, t, both(0.37409196f));
    p = fma2(p, t, both(1.00002368f));
    p = fma2(p, t, both(-1.26551223f));
    return t * exp2_fast(p * both(kLog2e));
}

// Phi(z), the normal distribution's function, and e^(-z^2 / 2).  The tail on
// the left is a small number of its own, not a difference of numbers near 1.
__device__ __forceinline__ Two normal_cdf(Two z, Two& e)
{
    const Two x = Two{fabsf(z.a), fabsf(z.b)} * both(0.70710678118654752f);
    e = exp2_fast(x * x * both(-kLog2e));
    const Two tail = e * erfc_factor(x) * both(0.5f);
    return {z.a < 0.0f ? tail.a : 1.0f - tail.a, z.b < 0.0f ? tail.b : 1.0f - tail.b};
}

// The logistic function's argument in gelu_tanh, times -log2(e); *square: z^2.
__device__ __forceinline__ Two gelu_tanh_exponent(Two z, Two* square)
{
    *square = z * z;
    return fma2(*square * both(kGeluA), z, z) * both(-2.0f * kGeluC * kLog2e);
}

template <int ACT>
__device__ __forceinline__ Two act_value(Two z)
{
    if constexpr (ACT == DRADD_ACT_RELU) {
        return {z.a < 0.0f ? 0.0f : z.a, z.b < 0.0f ? 0.0f : z.b};
    } else if constexpr (ACT == DRADD_ACT_GELU) {
        Two e;
        return z * normal_cdf(z, e);
    } else if constexpr (ACT == DRADD_ACT_GELU_TANH) {
        Two square;
        return z * logistic2(gelu_tanh_exponent(z, &square));
    } else {
        static_assert(ACT == DRADD_ACT_SILU);
        return z * logistic2(z * both(-kLog2e));
    }
}

// f + w z v: act'(z) of a product z f(z); where w has vanished, f alone,
// however large z is.
__device__ __forceinline__ Two slope_of(Two f, Two w, Two zv)
{
    const Two d = fma2(w, zv, f);
    return {w.a == 0.0f ? f.a : d.a, w.b == 0.0f ? f.b : d.b};
}

template <int ACT>
__device__ __forceinline__ Two act_slope(Two z)
{
    if constexpr (ACT == DRADD_ACT_RELU) {
        return {z.a > 0.0f ? 1.0f : 0.0f, z.b > 0.0f ? 1.0f : 0.0f};
    } else if constexpr (ACT == DRADD_ACT_GELU) {
        Two e;
        const Two f = normal_cdf(z, e);
        return slope_of(f, e, z * both(0.3989422804014327f));  // the normal density's factor
    } else if constexpr (ACT == DRADD_ACT_GELU_TANH) {
        Two square;
        const Two f = logistic2(gelu_tanh_exponent(z, &square));
        const Two w = fma2(f * both(-1.0f), f, f);
        return slope_of(f, w, z * fma2(square, both(6.0f * kGeluC * kGeluA), both(2.0f * kGeluC)));
    } else {
        static_assert(ACT == DRADD_ACT_SILU);
        const Two f = logistic2(z * both(-kLog2e));
        return slope_of(f, fma2(f * both(-1.0f), f, f), z);
    }
}

template <int ACT, int N>
__device__ __forceinline__ void act_values(float (&z)[N])
{
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const Two d = act_value<ACT>({z[j], N > 1 ? z[j + (N > 1)] : 0.0f});
        z[j] = d.a;
        if (N > 1)
            z[j + (N > 1)] = d.b;
    }
}

template <int ACT, int N>
__device__ __forceinline__ void act_slopes(float (&z)[N])
{
    static_assert(N % 2 == 0);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
        const Two d = act_slope<ACT>({z[j], z[j + 1]});
        z[j] = d.a;
        z[j + 1] = d.b;
    }
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
