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
    } else {
        static_assert(X == X_F32, "codes are read through LDS");
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

// The bf16 terms of a token matrix p [rows, R], laid out as the products with
// it read them: for each block of 16 rows, step by step of 32 slots, the 64
// lanes' eight values (lane l: row l % 16, slots 8 (l / 16) ..), so that a wave
// reads 1024 bytes in a row.  (Read row by row, every lane was a cache access of
// its own, and those took longer than the products.)  The form QT of the other
// operand decides the slots: 1, one bf16 term: p's three terms one after
// another, 3 R slots; 3, three terms: the six pairs of terms above 2^-24, the
// smallest first, 6 R slots; 0, fp32, split where it is used, and 4, three
// terms: the ranks in steps of 32, and each step once per term.  (3 is for the
// products' epilogues, whose registers hold one term of 64 columns at a time; 4
// is half its size.)
constexpr int terms_steps(int qt, int R)
{
    return qt == 0 || qt == 4 ? 3 * ((R + 31) / 32) : ((qt == 1 ? 3 : 6) * R + 31) / 32;
}

// Term of p in pair i of six (of the other operand: pair_other).
__host__ __device__ constexpr int pair_term(int i) { return (0x001012 >> (4 * i)) & 3; }
__host__ __device__ constexpr int pair_other(int i) { return (0x010210 >> (4 * i)) & 3; }

// Where slot k of a row lies among the rows' terms.
__device__ __forceinline__ int64_t term_at(int steps, int64_t row, int k)
{
    return (((row / 16) * steps + k / 32) * 64 + row % 16 + 16 * (k % 32 / 8)) * 8 + k % 8;
}

// Writes N consecutive values of a row, from rank r (a multiple of N; N
// divides 8), into the terms.
template <int N>
__device__ __forceinline__ void put_terms(uint16_t *terms, int qt, int R, int64_t row, int r, const float (&v0)[N])
{
    const int steps = terms_steps(qt, R);
    float v[N];
#pragma unroll
    for (int e = 0; e < N; e++)
        v[e] = v0[e];
#pragma unroll
    for (int t = 0; t < 3; t++) {
        uint16_t b[N];
#pragma unroll
        for (int e = 0; e < N; e++) {
            const uint32_t w = pack_bf16x2(v[e], 0.0f);
            b[e] = (uint16_t)w;
            v[e] = v[e] - bf16_lo(w);
        }
        auto put = [&](int k) {
            uint16_t *at = terms + term_at(steps, row, k);
            if constexpr (N == 4)
                *reinterpret_cast<i32x2 *>(at) =
                    i32x2{(int)(b[0] | (uint32_t)b[1] << 16), (int)(b[2] | (uint32_t)b[3] << 16)};
            else
                *at = b[0];
        };
        if (qt == 0 || qt == 4) {
            put((r / 32 * 3 + t) * 32 + r % 32);
        } else if (qt == 1) {
            put(t * R + r);
        } else {
#pragma unroll
            for (int i = 0; i < 6; i++)
                if (pair_term(i) == t)
                    put(i * R + r);
        }
    }
}

// Writes eight values of the other operand's three terms into their slots (of
// the six pairs, QT = 3, or QT = 4): column c, ranks r .. r + 7.
__device__ __forceinline__ void put_other(uint16_t *terms, int qt, int R, int64_t c, int r, const float (&v)[8])
{
    const int steps = terms_steps(qt, R);
    const Frag<3> f = split8(v);
    if (qt == 4) {
#pragma unroll
        for (int t = 0; t < 3; t++)
            *reinterpret_cast<bf16x8 *>(terms + term_at(steps, c, (r / 32 * 3 + t) * 32 + r % 32)) = f.t[t];
        return;
    }
#pragma unroll
    for (int i = 0; i < 6; i++)
        *reinterpret_cast<bf16x8 *>(terms + term_at(steps, c, i * R + r)) = f.t[pair_other(i)];
}

} // namespace

} // namespace qlin
