// AdamW over a list of float tensors in one launch, with fp32 moments or with
// moments in 8 bits (e4m3 codes with one fp32 scale per 256 elements).
//
//   m' = b1 m + a1 g         v' = b2 v + (a2 g) g        r' = sqrt(v')
//   p' = p (1 - lr wd) - c1 (m' / (r' c2 + eps))
//
// with a1 = 1 - b1, a2 = 1 - b2, c1 = lr / (1 - b1^t), c2 = 1 / sqrt(1 - b2^t).
//
// 8-bit moments.  The second moment is held as its root r: e4m3 spans 2^17 in
// r, hence 2^34 in v, inside one block.  Its codes are rounded stochastically:
// with b2 = 0.999 a step moves v by a part in a thousand, far less than half
// of an e4m3 step (1/16 to 1/8 of the value), so rounding to nearest would
// leave it where it is for good; a value above zero never becomes zero, or the
// next step would divide by eps alone.  The first moment moves by a tenth of
// the gradient's difference every step and is rounded to nearest.  bf16
// parameters are rounded stochastically too, for the same reason as v.  The
// arithmetic is fp32 throughout.
//
// A chunk of 4096 elements is one workgroup's work; a lane holds two runs of
// eight elements, and 16 lanes a block of 256, whose absmax is found with four
// DPP steps.  One read and one write of each array: the HBM traffic bounds it.
#include "common.hpp"
#include "launch.hpp"
#include "lowp.hpp"
#include "philox.hpp"
#include "tensors.hpp"

namespace qlin {

namespace {

constexpr float kTinyBlock = 0x1p-100f;     // blocks whose absmax is below hold zeros
constexpr float kE4m3Max = 448.0f;

struct StepArgs {
    const TensorEntry *tensors;
    const int32_t *chunk_tensor;
    float b1, b2, eps, a1, a2, c1, c2, lr;
    uint32_t seed_lo, seed_hi, step_lo, step_hi;
};

// Eight e4m3 codes at a byte pointer (8-byte aligned) as floats.
__device__ __forceinline__ void unpack_e4m3x8(i32x2 w, float v[8])
{
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
        v[4 * k] = lo[0];
        v[4 * k + 1] = lo[1];
        v[4 * k + 2] = hi[0];
        v[4 * k + 3] = hi[1];
    }
}

// Floats within +-448 (or NaN) as e4m3 codes, rounded to nearest even.
__device__ __forceinline__ i32x2 pack_e4m3x8(const float v[8])
{
    i32x2 w;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        int x = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k], v[4 * k + 1], 0, false);
        w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2], v[4 * k + 3], x, true);
    }
    return w;
}

// t in [0, 448] rounded to an e4m3 value, up with the probability that r16 /
// 2^16 gives: r16 is added below the last kept mantissa bit, then the rest is
// cut off.  Values below 2^-6 are e4m3 subnormals, multiples of 2^-9: adding
// 2^-6 gives them that last bit.
__device__ __forceinline__ float stochastic_e4m3(float t, uint32_t r16)
{
    const float low = t < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t bits = (__float_as_uint(t + low) + (r16 << 4)) & ~0xFFFFFu;
    const float near = __uint_as_float(bits) - low;
    return t > 0.0f ? fmaxf(near, 0x1p-9f) : near;
}

// The 16-bit uniforms of the eight elements from index 8 blk.
__device__ __forceinline__ void uniforms8(const StepArgs &a, uint64_t blk, uint32_t stream,
                                          uint32_t r[8])
{
    uint32_t x[4] = {(uint32_t)blk, (uint32_t)(blk >> 32), a.step_lo, a.step_hi + stream};
    philox4x32_10(x, a.seed_lo, a.seed_hi);
#pragma unroll
    for (int e = 0; e < 8; e++)
        r[e] = (x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
}

// Eight elements from 'idx' of an fp32 or bf16 array of n; those past its end
// read as zeros.
template <bool BF16>
__device__ __forceinline__ void load8_tail(const void *p, int64_t idx, int64_t n, float v[8])
{
    if (idx + 8 <= n) {
        load8<BF16>(p, idx, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        v[e] = 0.0f;
        if (idx + e < n) {
            if constexpr (BF16)
                v[e] = bf16_lo(static_cast<const uint16_t *>(p)[idx + e]);
            else
                v[e] = static_cast<const float *>(p)[idx + e];
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_tail(T *p, int64_t idx, int64_t n, const T v[8])
{
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (idx + e < n)
            p[idx + e] = v[e];
}

template <bool PB, bool GB, bool S8>
__device__ void step_chunk(const StepArgs &a, const TensorEntry &t, int64_t c0)
{
    constexpr int kRuns = 2;            // of eight elements per lane
    const int64_t n = t.numel;
    const float decay = __builtin_fmaf(-a.lr, t.weight_decay, 1.0f);
    // Lane l of 16 holds elements 8 l .. 8 l + 7 and 128 + 8 l .. of its block.
    const int64_t at = c0 + (threadIdx.x / 16) * kStateBlock + (threadIdx.x % 16) * 8;
    const int64_t blk = at / kStateBlock;
    if (at >= n && !S8)
        return;
    float p[kRuns][8], g[kRuns][8], m[kRuns][8], v[kRuns][8];
    float sm = 0.0f, sv = 0.0f;
    if (S8 && blk * kStateBlock < n) {
        sm = t.ms[blk];
        sv = t.vs[blk];
    }
#pragma unroll
    for (int k = 0; k < kRuns; k++) {
        const int64_t i = at + 128 * k;
        load8_tail<PB>(t.p, i, n, p[k]);
        load8_tail<GB>(t.g, i, n, g[k]);
        if constexpr (S8) {
            i32x2 wm = {0, 0}, wv = {0, 0};
            if (i + 8 <= n) {
                wm = *reinterpret_cast<const i32x2 *>(static_cast<const uint8_t *>(t.m) + i);
                wv = *reinterpret_cast<const i32x2 *>(static_cast<const uint8_t *>(t.v) + i);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (i + e < n) {
                        wm[e / 4] |= static_cast<const uint8_t *>(t.m)[i + e] << (8 * (e % 4));
                        wv[e / 4] |= static_cast<const uint8_t *>(t.v)[i + e] << (8 * (e % 4));
                    }
            }
            unpack_e4m3x8(wm, m[k]);
            unpack_e4m3x8(wv, v[k]);
        } else {
            load8_tail<false>(t.m, i, n, m[k]);
            load8_tail<false>(t.v, i, n, v[k]);
        }
    }
    float am = 0.0f, av = 0.0f;
#pragma unroll
    for (int k = 0; k < kRuns; k++) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (S8) {
                m[k][e] = m[k][e] * sm;
                const float r = v[k][e] * sv;
                v[k][e] = r * r;
            }
            m[k][e] = a.b1 * m[k][e] + a.a1 * g[k][e];
            v[k][e] = a.b2 * v[k][e] + (a.a2 * g[k][e]) * g[k][e];
            const float r = __builtin_sqrtf(v[k][e]);
            p[k][e] = p[k][e] * decay - a.c1 * (m[k][e] / __builtin_fmaf(r, a.c2, a.eps));
            if constexpr (S8) {
                v[k][e] = r;
                am = max_nan(am, __builtin_fabsf(m[k][e]));
                av = max_nan(av, r);
            }
        }
    }
    float im = 0.0f, iv = 0.0f;
    if constexpr (S8) {
        auto most = [](float x, float y) { return max_nan(x, y); };
        am = row16_all(am, most);
        av = row16_all(av, most);
        // (A NaN is kept: it makes the block's scale NaN.)
        const bool zm = am < kTinyBlock, zv = av < kTinyBlock;
        im = zm ? 0.0f : (1.0f / am) * kE4m3Max;
        iv = zv ? 0.0f : (1.0f / av) * kE4m3Max;
        if (threadIdx.x % 16 == 0 && blk * kStateBlock < n) {
            t.ms[blk] = zm ? 0.0f : am * (1.0f / kE4m3Max);
            t.vs[blk] = zv ? 0.0f : av * (1.0f / kE4m3Max);
        }
    }
#pragma unroll
    for (int k = 0; k < kRuns; k++) {
        const int64_t i = at + 128 * k;
        if (i >= n)
            continue;
        const bool whole = i + 8 <= n;
        const uint64_t u = (uint64_t)(t.index0 + i) >> 3;
        if constexpr (PB) {
            uint32_t r[8];
            uniforms8(a, u, 0x80000000u, r);
            uint16_t o[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const uint32_t b = __float_as_uint(p[k][e]);
                // (Adding to an infinity's or a NaN's bits would change which it is.)
                const bool finite = (b & 0x7F800000u) != 0x7F800000u;
                o[e] = (uint16_t)((finite ? b + r[e] : b) >> 16);
            }
            uint16_t *dst = static_cast<uint16_t *>(t.p);
            if (whole) {
                i32x4 w;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[e] = (int)(o[2 * e] | (uint32_t)o[2 * e + 1] << 16);
                *reinterpret_cast<i32x4 *>(dst + i) = w;
            } else {
                store_tail(dst, i, n, o);
            }
        } else if (whole) {
            store8(static_cast<float *>(t.p), i, p[k]);
        } else {
            store_tail(static_cast<float *>(t.p), i, n, p[k]);
        }
        if constexpr (S8) {
            uint32_t r[8];
            uniforms8(a, u, 0u, r);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                // (A block with a NaN has a NaN scale; its codes do not matter.)
                m[k][e] = fminf(fmaxf(m[k][e] * im, -kE4m3Max), kE4m3Max);
                v[k][e] = stochastic_e4m3(fminf(v[k][e] * iv, kE4m3Max), r[e]);
            }
            const i32x2 wm = pack_e4m3x8(m[k]), wv = pack_e4m3x8(v[k]);
            uint8_t *dm = static_cast<uint8_t *>(t.m), *dv = static_cast<uint8_t *>(t.v);
            if (whole) {
                *reinterpret_cast<i32x2 *>(dm + i) = wm;
                *reinterpret_cast<i32x2 *>(dv + i) = wv;
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (i + e < n) {
                        dm[i + e] = (uint8_t)((uint32_t)wm[e / 4] >> (8 * (e % 4)));
                        dv[i + e] = (uint8_t)((uint32_t)wv[e / 4] >> (8 * (e % 4)));
                    }
            }
        } else if (whole) {
            store8(static_cast<float *>(t.m), i, m[k]);
            store8(static_cast<float *>(t.v), i, v[k]);
        } else {
            store_tail(static_cast<float *>(t.m), i, n, m[k]);
            store_tail(static_cast<float *>(t.v), i, n, v[k]);
        }
    }
}

__global__ __launch_bounds__(256) void adamw_tensors_kernel(StepArgs a)
{
    const TensorEntry t = a.tensors[a.chunk_tensor[blockIdx.x]];
    const int64_t c0 = ((int64_t)blockIdx.x - t.chunk0) * kTensorChunk;
    switch (t.flags) {
    case 0: return step_chunk<false, false, false>(a, t, c0);
    case 1: return step_chunk<true, false, false>(a, t, c0);
    case 2: return step_chunk<false, true, false>(a, t, c0);
    case 3: return step_chunk<true, true, false>(a, t, c0);
    case 4: return step_chunk<false, false, true>(a, t, c0);
    case 5: return step_chunk<true, false, true>(a, t, c0);
    case 6: return step_chunk<false, true, true>(a, t, c0);
    default: return step_chunk<true, true, true>(a, t, c0);
    }
}

} // namespace

void launch_adamw_tensors(const void *image, int64_t count, int64_t chunks, const AdamTensorConsts &k,
                          uint64_t seed, uint64_t step, hipStream_t st)
{
    StepArgs a;
    a.tensors = static_cast<const TensorEntry *>(image);
    a.chunk_tensor = reinterpret_cast<const int32_t *>(a.tensors + count);
    a.b1 = k.b1;
    a.b2 = k.b2;
    a.eps = k.eps;
    a.a1 = k.a1;
    a.a2 = k.a2;
    a.c1 = k.c1;
    a.c2 = k.c2;
    a.lr = k.lr;
    a.seed_lo = (uint32_t)seed;
    a.seed_hi = (uint32_t)(seed >> 32);
    a.step_lo = (uint32_t)step;
    a.step_hi = (uint32_t)(step >> 32);
    hipLaunchKernelGGL(adamw_tensors_kernel, dim3((unsigned)chunks), dim3(256), 0, st, a);
}

} // namespace qlin
