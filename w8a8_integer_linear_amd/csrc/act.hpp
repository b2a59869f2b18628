// Activations between the projections of a feed-forward block, and their
// derivatives, in fp32 (values and slopes share their transcendental parts).
//
//   silu       z s(z), s the logistic function
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z s(2 sqrt(2/pi) (z + 0.044715 z^3)), the same as
//              z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
//
// The logistic function is 1 / (1 + 2^(-z log2 e)) by the hardware's exp2 and
// reciprocal (1 ulp each): a relative error of about 2^-22 plus 2^-24 |z| from
// the rounded exponent, the latter where s(z) is small.
//
// Phi in two forms, both without a branch (the library's erf has two, of which a wave
// takes both):
//   normal_cdf, for the derivative, which needs e^(-z^2/2) beside it: Phi(-x), x >= 0,
//   is that times a polynomial of degree 8 without a constant term in t = 1 / (1 +
//   0.3 x); erfc's scaled form is smooth in t and falls like t for large x.  Relative
//   error at most 1.3e-7 over 0 <= x <= 14, past which the exponential is below 2^-126.
//   gelu_value, for the value alone: z Phi(z) = max(z, 0) - x Phi(-x), x = |z|, with
//   Phi(-x) = 2^P(x), P of degree 7 (log2 of Phi is nearly a parabola).  x 2^P(x) is
//   within 4.7e-8 for x <= 6, and taken at 6, where it is 5.9e-9, past that.  One
//   transcendental instruction instead of two: 14 issue slots against 25, and the
//   product's epilogue is bound by those (4000 x 4096 -> 14336 with it: 229 -> 219 us).
// The coefficients are minimax fits (linear programming) of these errors.
#pragma once

#include <hip/hip_runtime.h>

#include "qlin.h"

namespace qlin {

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// s(z); 0 where the exponential overflows.
__device__ __forceinline__ float logistic(float z) { return rcp_hw(1.0f + exp2_hw(z * -kLog2e)); }

// Phi(z), and e^(-z^2/2).
__device__ __forceinline__ float normal_cdf(float z, float &gauss)
{
    const float x = __builtin_fabsf(z);
    const float t = rcp_hw(__builtin_fmaf(x, 0.3f, 1.0f));
    gauss = exp2_hw(z * z * (-0.5f * kLog2e));
    float q = 0.03556719721f;
    q = __builtin_fmaf(q, t, -0.156760921f);
    q = __builtin_fmaf(q, t, 0.2056028133f);
    q = __builtin_fmaf(q, t, -0.05300297223f);
    q = __builtin_fmaf(q, t, 0.1282069439f);
    q = __builtin_fmaf(q, t, 0.1000190791f);
    q = __builtin_fmaf(q, t, 0.1207374586f);
    q = __builtin_fmaf(q, t, 0.1196303368f);
    q = q * t * gauss;
    return z < 0.0f ? q : 1.0f - q;
}

__device__ __forceinline__ float gelu_value(float z)
{
    const float x = __builtin_elementwise_minimum(__builtin_fabsf(z), 6.0f);
    float q = 3.304236914e-06f;
    q = __builtin_fmaf(q, x, -4.404308744e-06f);
    q = __builtin_fmaf(q, x, -0.0006028252271f);
    q = __builtin_fmaf(q, x, 0.007711402484f);
    q = __builtin_fmaf(q, x, -0.05297750938f);
    q = __builtin_fmaf(q, x, -0.459034572f);
    q = __builtin_fmaf(q, x, -1.151128862f);
    q = __builtin_fmaf(q, x, -0.9999994886f);
    return __builtin_fmaf(-x, exp2_hw(q), fmaxf(z, 0.0f));
}

constexpr float kTanhRate = 1.5957691216f;      // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

__device__ __forceinline__ float tanh_inner(float z)
{
    return z * __builtin_fmaf(z * z, kTanhRate * kTanhCube, kTanhRate);
}

template <int ACT> __device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == QLIN_ACT_RELU) {
        return z > 0.0f || z != z ? z : 0.0f;
    } else if constexpr (ACT == QLIN_ACT_SILU) {
        return z * logistic(z);
    } else if constexpr (ACT == QLIN_ACT_GELU) {
        return gelu_value(z);
    } else if constexpr (ACT == QLIN_ACT_GELU_TANH) {
        return z * logistic(tanh_inner(z));
    } else {
        return z;
    }
}

// The value and the derivative.
template <int ACT> __device__ __forceinline__ void act_slope(float z, float &value, float &slope)
{
    if constexpr (ACT == QLIN_ACT_RELU) {
        value = act_value<ACT>(z);
        slope = z > 0.0f ? 1.0f : z != z ? z : 0.0f;
    } else if constexpr (ACT == QLIN_ACT_SILU) {
        const float s = logistic(z);
        value = z * s;
        slope = __builtin_fmaf(value, 1.0f - s, s);
    } else if constexpr (ACT == QLIN_ACT_GELU) {
        float gauss;
        const float cdf = normal_cdf(z, gauss);
        value = z * cdf;
        slope = __builtin_fmaf(z * 0.3989422804f, gauss, cdf);
    } else if constexpr (ACT == QLIN_ACT_GELU_TANH) {
        const float s = logistic(tanh_inner(z));
        value = z * s;
        const float rate = __builtin_fmaf(z * z, 3.0f * kTanhRate * kTanhCube, kTanhRate);
        slope = __builtin_fmaf(value * (1.0f - s), rate, s);
    } else {
        value = z;
        slope = 1.0f;
    }
}

} // namespace qlin
