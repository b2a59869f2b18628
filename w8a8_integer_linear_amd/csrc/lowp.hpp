// Device helpers of the norm, adapter and optimizer kernels: bf16 and e4m3
// conversions, NaN-keeping maxima, wave reductions and the Philox generator.
#pragma once

#include "common.hpp"

namespace qlin {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Two floats rounded to bf16 (nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

__device__ __forceinline__ i32x4 pack_bf16x8(const float v[8])
{
    i32x4 w;
#pragma unroll
    for (int e = 0; e < 4; e++)
        w[e] = (int)pack_bf16x2(v[2 * e], v[2 * e + 1]);
    return w;
}

// Eight INT8 codes as floats.
__device__ __forceinline__ void codes_to_float(i32x2 q, float v[8])
{
#pragma unroll
    for (int e = 0; e < 8; e++)
        v[e] = (float)(int8_t)(uint8_t)((uint32_t)q[e / 4] >> (8 * (e % 4)));
}

// Maximum that is NaN if either operand is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    return __builtin_elementwise_maximum(a, b);
}

// Reduction over 16 lanes (aligned), every lane gets the result: partners
// lane ^ 1 and ^ 2 by quad permutes, then the half row's and the row's mirror
// images.  op is commutative, so partners compute the same bits.
template <typename Op>
__device__ __forceinline__ float row16_all(float v, Op op)
{
    v = op(v, dpp_mov<0xB1>(v));
    v = op(v, dpp_mov<0x4E>(v));
    v = op(v, dpp_mov<0x141>(v));
    v = op(v, dpp_mov<0x140>(v));
    return v;
}

// Reduction over the wave, every lane gets the result.
template <typename Op>
__device__ __forceinline__ float wave_all(float v, Op op)
{
    v = row16_all(v, op);
    const uint32_t x = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const uint32_t y = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return op(__uint_as_float(h[0]), __uint_as_float(h[1]));
}

} // namespace qlin
