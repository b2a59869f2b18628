// Activations between the projections of a feed-forward block, and their
// derivatives, in fp32 (values and slopes share their transcendental parts).
//
//   silu       z s(z), s the logistic function
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  z s(2 sqrt(2/pi) (z + 0.044715 z^3)), the same as
//              z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
//
// The logistic function is 1 / (1 + 2^(-z log2 e)) by the hardware's exp2 and
// reciprocal (1 ulp each): a relative error of about 2^-22 plus 1.3 2^-24 |z| from
// the rounded exponent and its constant, the latter where s(z) is small.
//
// Phi without a branch (the library's erf has two, of which a wave takes both): for x =
// |z|, Phi(-x) is e^(-x^2/2) times a polynomial of degree 9 without a constant term in t =
// 1 / (1 + 0.34 x); erfc's scaled form is smooth in t and falls like t for large x.  The
// coefficients are a minimax fit (linear programming) of the relative error, each rounded
// to fp32 before the next is fitted: 4.1e-8 over 0 <= x <= 13.2, past which the
// exponential is below 2^-126 and may be flushed.  As computed in fp32, Phi(-x) is within
// 4.5e-7 of itself for x <= 2, and within 2^-21 + 2^-24 x^2 further out, where the rounded
// exponent is what counts (2.1e-6 at 6).
//   z Phi(z) = max(z, 0) - x Phi(-x), with x = min(|z|, 20), where the exponential is 0.
// Forward and backward take this one form.  (A polynomial P of degree 7 with Phi(-x) =
// 2^P(x) has one transcendental instruction instead of two, 14 issue slots against 24, but
// only an absolute error: 5% of the value at -6, a constant below.  us, that / this: 4000 x
// 4096 -> 14336 with checkpoint and backward 326 / 337, 777 x 4096 -> 14336 59.7 / 61.3.)
#pragma once

#include <hip/hip_runtime.h>

#include "qlin.h"

namespace qlin {

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// s(z); 0 where the exponential overflows.
__device__ __forceinline__ float logistic(float z) { return rcp_hw(1.0f + exp2_hw(z * -kLog2e)); }

// Phi(-x) and e^(-x^2/2), x >= 0.
__device__ __forceinline__ float normal_tail(float x, float &gauss)
{
    const float t = rcp_hw(__builtin_fmaf(x, 0.34f, 1.0f));
    gauss = exp2_hw(x * x * (-0.5f * kLog2e));
    float q = -0.02649738826f;
    q = __builtin_fmaf(q, t, 0.141270116f);
    q = __builtin_fmaf(q, t, -0.2766533494f);
    q = __builtin_fmaf(q, t, 0.2060405612f);
    q = __builtin_fmaf(q, t, -0.04725845158f);
    q = __builtin_fmaf(q, t, 0.1163846999f);
    q = __builtin_fmaf(q, t, 0.1149504483f);
    q = __builtin_fmaf(q, t, 0.1361446381f);
    q = __builtin_fmaf(q, t, 0.1356187314f);
    return q * t * gauss;
}

// z Phi(z), and what its derivative needs: Phi(-x) and e^(-x^2/2).
__device__ __forceinline__ float gelu(float z, float &tail, float &gauss)
{
    const float x = __builtin_elementwise_minimum(__builtin_fabsf(z), 20.0f);
    tail = normal_tail(x, gauss);
    return __builtin_fmaf(-x, tail, fmaxf(z, 0.0f));
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
        float tail, gauss;
        return gelu(z, tail, gauss);
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
        float tail, gauss;
        value = gelu(z, tail, gauss);
        slope = __builtin_fmaf(z * 0.3989422804f, gauss, z < 0.0f ? tail : 1.0f - tail);
    } else if constexpr (ACT == QLIN_ACT_GELU_TANH) {
        const float s = logistic(tanh_inner(z));
        value = z * s;
        // (A finite rate: z^2 passes fp32 at 2^64, where 1 - s or the value is 0.)
        const float rate = __builtin_fmaf(fminf(z * z, 0x1p64f), 3.0f * kTanhRate * kTanhCube, kTanhRate);
        slope = __builtin_fmaf(value * (1.0f - s), rate, s);
    } else {
        value = z;
        slope = 1.0f;
    }
}

} // namespace qlin
