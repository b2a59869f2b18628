// Operands of the adapters' products on v_mfma_f32_16x16x32_bf16: INT8 codes
// and bf16 as they are, fp32 split into three bf16 terms.
#pragma once

#include "common.hpp"
#include "lowp.hpp"

namespace qlin {

namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

enum { X_I8 = 0, X_BF16 = 1, X_F32 = 2 };

// An MFMA operand: eight contraction values per lane, as one or three bf16
// terms, each the rounded rest that the ones before it leave.
template <int TERMS> struct Frag {
    bf16x8 t[TERMS];
};

__device__ __forceinline__ bf16x8 zero8() { return __builtin_bit_cast(bf16x8, i32x4{0, 0, 0, 0}); }

__device__ __forceinline__ bf16x8 round8(const float v[8])
{
    return __builtin_bit_cast(bf16x8, pack_bf16x8(v));
}

__device__ __forceinline__ Frag<3> split8(const float v[8])
{
    Frag<3> f;
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; e++)
        rest[e] = v[e];
#pragma unroll
    for (int q = 0; q < 3; q++) {
        f.t[q] = round8(rest);
        if (q < 2) {
            float t[8];
            unpack8<true>(Raw8<true>{__builtin_bit_cast(i32x4, f.t[q])}, t);
#pragma unroll
            for (int e = 0; e < 8; e++)
                rest[e] = rest[e] - t[e];
        }
    }
    return f;
}

constexpr int terms_of(int x) { return x == X_F32 ? 3 : 1; }

// Eight consecutive elements from index idx (a multiple of 8); zeros unless ok.
template <int X>
__device__ __forceinline__ Frag<terms_of(X)> load_frag(const void *p, int64_t idx, bool ok)
{
    Frag<terms_of(X)> f;
    if constexpr (X == X_BF16) {
        f.t[0] = zero8();
        if (ok)
            f.t[0] = *reinterpret_cast<const bf16x8 *>(static_cast<const uint16_t *>(p) + idx);
        return f;
    } else if constexpr (X == X_I8) {
        i32x2 w = {0, 0};
        if (ok)
            w = *reinterpret_cast<const i32x2 *>(static_cast<const int8_t *>(p) + idx);
        float v[8];
        codes_to_float(w, v);
        f.t[0] = round8(v);
        return f;
    } else {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (ok)
            load8<false>(p, idx, v);
        return split8(v);
    }
}

// acc += a b over the terms, the smallest first; of nine partial products of
// two split operands, the three below 2^-24 are left out.
template <int TA, int TB>
__device__ __forceinline__ f32x4 mfma(const Frag<TA> &a, const Frag<TB> &b, f32x4 acc)
{
#pragma unroll
    for (int d = 2; d >= 0; d--)
#pragma unroll
        for (int i = 0; i < TA; i++)
            if (d - i >= 0 && d - i < TB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.t[i], b.t[d - i], acc, 0, 0, 0);
    return acc;
}

// f(id, mine) for every adapter among the wave's 16 tokens (lane l holds token
// l % 16's id, or -1); mine: whether this lane's token has it.
template <typename F> __device__ __forceinline__ void for_adapters(int id, F f)
{
    uint64_t left = __ballot(id >= 0);
    while (left) {
        const int cur = __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(left));
        const bool mine = id == cur;
        f(cur, mine);
        left &= ~__ballot(mine);
    }
}

__device__ __forceinline__ int id_of(const int32_t *ids, int64_t m, int64_t M, int L)
{
    const int id = m < M ? ids[m] : -1;
    return id >= 0 && id < L ? id : -1;
}

} // namespace

} // namespace qlin
