// AdamW over a list of float tensors in one launch, with fp32 moments or with
// moments in 8 bits (e4m3 codes with one fp32 scale per 256 elements).
//
//   m' = b1 m + a1 g         v' = b2 v + (a2 g) g        r' = sqrt(v')
//   p' = p (1 - lr wd) - c1 (m' / (r' c2 + eps))
//
// with a1 = 1 - b1, a2 = 1 - b2, c1 = lr / (1 - b1^t), c2 = 1 / sqrt(1 - b2^t); c1,
// c2 and eps come times 2^24, which the quotient leaves as it is.
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
// DPP steps.  One read and one write of each array: the HBM traffic bounds it
// (fp32 moments, 1.98 GB: 359 us; 8 bits, 1.61 GB: 295 us; both 5.5 TB/s, where a
// streaming copy of 1 GiB reaches 6.2).
#include <type_traits>

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
    const int32_t *chunk_tensor;        // of the launch's chunks
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

// Eight values t in [0, 448] as e4m3 codes, each rounded up with the
// probability that its place between two codes gives: the conversion adds the
// uniform r16 / 2^16 (seed = r16 << 16) below the last kept bit and cuts off.
// A value above zero gets at least the smallest code, 2^-9: the median of t,
// 2^-9 and 2^100 t is 0 for 0, 2^-9 below 2^-9 and t above.
__device__ __forceinline__ i32x2 stochastic_e4m3x8(const float t[8], const uint32_t x[4])
{
    i32x2 w = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; h++) {
        int c = 0;
        auto put = [&](auto E) {
            constexpr int e = decltype(E)::value;
            const float v = t[4 * h + e];
            const uint32_t word = x[2 * h + e / 2];
            const uint32_t seed = e % 2 ? word & 0xFFFF0000u : word << 16;
            c = __builtin_amdgcn_cvt_sr_fp8_f32(
                __builtin_amdgcn_fmed3f(v, 0x1p-9f, v * 0x1p100f), (int)seed, c, e);
        };
        put(std::integral_constant<int, 0>{});
        put(std::integral_constant<int, 1>{});
        put(std::integral_constant<int, 2>{});
        put(std::integral_constant<int, 3>{});
        w[h] = c;
    }
    return w;
}

// The 16-bit uniforms of the eight elements from index 8 blk, two per word.
__device__ __forceinline__ void uniforms8(const StepArgs &a, uint64_t blk, uint32_t stream,
                                          uint32_t x[4])
{
    x[0] = (uint32_t)blk;
    x[1] = (uint32_t)(blk >> 32);
    x[2] = a.step_lo;
    x[3] = a.step_hi + stream;
    philox4x32_10(x, a.seed_lo, a.seed_hi);
}

// Eight floats as bf16, rounded stochastically with the uniforms x; infinities
// and NaN (which adding to the bits would turn into one another) as they are.
__device__ __forceinline__ i32x4 stochastic_bf16x8(const float v[8], const uint32_t x[4])
{
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++)
        top = max_nan(top, __builtin_fabsf(v[e]));
    const bool finite = top < __builtin_inff();
    i32x4 w;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        uint32_t lo = __float_as_uint(v[2 * e]) + (x[e] & 0xFFFFu);
        uint32_t hi = __float_as_uint(v[2 * e + 1]) + (x[e] >> 16);
        if (!finite) {
            lo = __builtin_fabsf(v[2 * e]) < __builtin_inff() ? lo : __float_as_uint(v[2 * e]);
            hi = __builtin_fabsf(v[2 * e + 1]) < __builtin_inff() ? hi : __float_as_uint(v[2 * e + 1]);
            // a NaN stays one when its low half is cut off
            lo |= v[2 * e] != v[2 * e] ? 0x400000u : 0u;
            hi |= v[2 * e + 1] != v[2 * e + 1] ? 0x400000u : 0u;
        }
        w[e] = (int)__builtin_amdgcn_perm(hi, lo, 0x07060302u);
    }
    return w;
}

// sqrt(v) within half an ulp and a relative 2^-46, for every v of a lane in
// [2^-96, 2^96]: the hardware's reciprocal root and one correction of s = v y
// by (v - s^2) y / 2 (eight issue slots against seventeen for the correctly
// rounded root).  Other values take the correctly rounded root.
template <int N> __device__ __forceinline__ void roots(const float v[N], float r[N])
{
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int e = 1; e < N; e++) {
        lo = fminf(lo, v[e]);
        hi = fmaxf(hi, v[e]);
    }
    if (lo >= 0x1p-96f && hi <= 0x1p96f) {
#pragma unroll
        for (int e = 0; e < N; e++) {
            const float y = __builtin_amdgcn_rsqf(v[e]), s = v[e] * y;
            r[e] = __builtin_fmaf(__builtin_fmaf(-s, s, v[e]), 0.5f * y, s);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; e++)
            r[e] = __builtin_sqrtf(v[e]);
    }
}

// Global memory at a pointer that was itself read from memory (the compiler
// would take it for a generic one and use flat accesses).
template <typename T> __device__ __forceinline__ T gload(const void *p, int64_t byte)
{
    typedef const __attribute__((address_space(1))) T *G;
    return *(G)(uintptr_t)(static_cast<const char *>(p) + byte);
}
template <typename T> __device__ __forceinline__ void gstore(void *p, int64_t byte, T v)
{
    typedef __attribute__((address_space(1))) T *G;
    *(G)(uintptr_t)(static_cast<char *>(p) + byte) = v;
}

// Eight elements from 'idx' of an fp32 or bf16 array of n; those past its end
// read as zeros.  WHOLE: there are none.
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void load_eight(const void *p, int64_t idx, int64_t n, float v[8])
{
    if (WHOLE || idx + 8 <= n) {
        Raw8<BF16> r;
        if constexpr (BF16) {
            r.w = gload<i32x4>(p, idx * 2);
        } else {
            r.a = gload<f32x4>(p, idx * 4);
            r.b = gload<f32x4>(p, idx * 4 + 16);
        }
        unpack8<BF16>(r, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        v[e] = 0.0f;
        if (idx + e < n) {
            if constexpr (BF16)
                v[e] = bf16_lo(gload<uint16_t>(p, (idx + e) * 2));
            else
                v[e] = gload<float>(p, (idx + e) * 4);
        }
    }
}

template <bool WHOLE>
__device__ __forceinline__ void store_eight(void *p, int64_t idx, int64_t n, const float v[8])
{
    if (WHOLE || idx + 8 <= n) {
        gstore(p, idx * 4, f32x4{v[0], v[1], v[2], v[3]});
        gstore(p, idx * 4 + 16, f32x4{v[4], v[5], v[6], v[7]});
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (idx + e < n)
            gstore(p, (idx + e) * 4, v[e]);
}

// Eight one-byte codes.
template <bool WHOLE>
__device__ __forceinline__ i32x2 load_codes(const void *p, int64_t idx, int64_t n)
{
    if (WHOLE || idx + 8 <= n)
        return gload<i32x2>(p, idx);
    i32x2 w = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (idx + e < n)
            w[e / 4] |= gload<uint8_t>(p, idx + e) << (8 * (e % 4));
    return w;
}

template <bool WHOLE>
__device__ __forceinline__ void store_codes(void *p, int64_t idx, int64_t n, i32x2 w)
{
    if (WHOLE || idx + 8 <= n) {
        gstore(p, idx, w);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (idx + e < n)
            gstore(p, idx + e, (uint8_t)((uint32_t)w[e / 4] >> (8 * (e % 4))));
}

// WHOLE: the chunk ends before the tensor does, so nothing is checked.
template <bool PB, bool GB, bool S8, bool WHOLE>
__device__ __forceinline__ void step_chunk(const StepArgs &a, const TensorEntry &t, int64_t c0)
{
    constexpr int kRuns = 2;            // of eight elements per lane
    const int64_t n = t.numel;
    const float decay = __builtin_fmaf(-a.lr, t.weight_decay, 1.0f);
    // Lane l of 16 holds elements 8 l .. 8 l + 7 and 128 + 8 l .. of its block.
    const int64_t at = c0 + (threadIdx.x / 16) * kStateBlock + (threadIdx.x % 16) * 8;
    const int64_t blk = at / kStateBlock;
    const bool live = WHOLE || blk * kStateBlock < n;
    if (!live)                          // (all 16 lanes of a block agree)
        return;
    float p[kRuns][8], g[kRuns][8], m[kRuns][8], v[kRuns][8];
    i32x2 wm[kRuns], wv[kRuns];
    float sm = 0.0f, sv = 0.0f;
    if constexpr (S8) {
        sm = gload<float>(t.ms, blk * 4);
        sv = gload<float>(t.vs, blk * 4);
    }
#pragma unroll
    for (int k = 0; k < kRuns; k++) {
        const int64_t i = at + 128 * k;
        load_eight<PB, WHOLE>(t.p, i, n, p[k]);
        load_eight<GB, WHOLE>(t.g, i, n, g[k]);
        if constexpr (S8) {
            wm[k] = load_codes<WHOLE>(t.m, i, n);
            wv[k] = load_codes<WHOLE>(t.v, i, n);
        } else {
            load_eight<false, WHOLE>(t.m, i, n, m[k]);
            load_eight<false, WHOLE>(t.v, i, n, v[k]);
        }
    }
    float am = 0.0f, av = 0.0f;
#pragma unroll
    for (int k = 0; k < kRuns; k++) {
        if constexpr (S8) {
            unpack_e4m3x8(wm[k], m[k]);
            unpack_e4m3x8(wv[k], v[k]);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                m[k][e] = m[k][e] * sm;
                v[k][e] = v[k][e] * sv;
                v[k][e] = v[k][e] * v[k][e];
            }
        }
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            m[k][e] = a.b1 * m[k][e] + a.a1 * g[k][e];
            v[k][e] = a.b2 * v[k][e] + (a.a2 * g[k][e]) * g[k][e];
        }
        roots<8>(v[k], r);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            // (The quotient within about two ulps: it moves p by a part in 2^22
            // of the step.)
            p[k][e] = p[k][e] * decay -
                      a.c1 * (m[k][e] * __builtin_amdgcn_rcpf(__builtin_fmaf(r[e], a.c2, a.eps)));
            if constexpr (S8) {
                v[k][e] = r[e];
                am = max_nan(am, __builtin_fabsf(m[k][e]));
                av = max_nan(av, r[e]);
            }
        }
    }
    float im = 0.0f, iv = 0.0f;
    if constexpr (S8) {
        auto most = [](float x, float y) { return max_nan(x, y); };
        am = row16_all(am, most);
        av = row16_all(av, most);
        // A block with a NaN or an infinity gets a NaN scale: 448 / inf would leave
        // its finite values as zeros, which times an infinite scale are NaN, but one
        // step later and with a scale that does not say so.
        auto scale_of = [](float top, float &inv) {
            const bool zero = top < kTinyBlock;
            inv = zero ? 0.0f : (1.0f / top) * kE4m3Max;
            return zero ? 0.0f : top < __builtin_inff() ? top * (1.0f / kE4m3Max) : __builtin_nanf("");
        };
        const float cm = scale_of(am, im), cv = scale_of(av, iv);
        if (threadIdx.x % 16 == 0) {
            gstore(t.ms, blk * 4, cm);
            gstore(t.vs, blk * 4, cv);
        }
    }
#pragma unroll
    for (int k = 0; k < kRuns; k++) {
        const int64_t i = at + 128 * k;
        if (!WHOLE && i >= n)
            continue;
        const uint64_t u = (uint64_t)(t.index0 + i) >> 3;
        if constexpr (PB) {
            uint32_t x[4];
            uniforms8(a, u, 0x80000000u, x);
            const i32x4 w = stochastic_bf16x8(p[k], x);
            if (WHOLE || i + 8 <= n) {
                gstore(t.p, i * 2, w);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (i + e < n)
                        gstore(t.p, (i + e) * 2, (uint16_t)((uint32_t)w[e / 2] >> (16 * (e % 2))));
            }
        } else {
            store_eight<WHOLE>(t.p, i, n, p[k]);
        }
        if constexpr (S8) {
            // (The largest value's product with 448 / a may exceed 448 by a few
            // ulps; both conversions still give 448.  The codes of a block with
            // a NaN scale do not matter.)
            uint32_t x[4];
            uniforms8(a, u, 0u, x);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                m[k][e] = m[k][e] * im;
                v[k][e] = v[k][e] * iv;
            }
            store_codes<WHOLE>(t.m, i, n, pack_e4m3x8(m[k]));
            store_codes<WHOLE>(t.v, i, n, stochastic_e4m3x8(v[k], x));
        } else {
            store_eight<WHOLE>(t.m, i, n, m[k]);
            store_eight<WHOLE>(t.v, i, n, v[k]);
        }
    }
}

template <bool PB, bool GB, bool S8>
__device__ __forceinline__ void step_either(const StepArgs &a, const TensorEntry &t, int64_t c0)
{
    if (c0 + kTensorChunk <= t.numel)
        step_chunk<PB, GB, S8, true>(a, t, c0);
    else
        step_chunk<PB, GB, S8, false>(a, t, c0);
}

__device__ __forceinline__ void step_tensors(const StepArgs &a, uint32_t chunk0)
{
    const TensorEntry t = a.tensors[a.chunk_tensor[blockIdx.x]];
    const int64_t c0 = ((int64_t)(chunk0 + blockIdx.x) - t.chunk0) * kTensorChunk;
    switch (t.flags) {
    case 0: return step_either<false, false, false>(a, t, c0);
    case 1: return step_either<true, false, false>(a, t, c0);
    case 2: return step_either<false, true, false>(a, t, c0);
    case 3: return step_either<true, true, false>(a, t, c0);
    case 4: return step_either<false, false, true>(a, t, c0);
    case 5: return step_either<true, false, true>(a, t, c0);
    case 6: return step_either<false, true, true>(a, t, c0);
    default: return step_either<true, true, true>(a, t, c0);
    }
}

static_assert(sizeof(StepArgs) == 64, "the arguments are one cache line");

__global__ __launch_bounds__(256) void adamw_tensors_kernel(StepArgs a) { step_tensors(a, 0); }

// The same from chunk chunk0 on, for lists that take several launches.  (A kernel of
// its own: the argument past the first 64 bytes costs a short list 0.35 us of 17.)
__global__ __launch_bounds__(256) void adamw_tensors_from_kernel(StepArgs a, uint32_t chunk0)
{
    step_tensors(a, chunk0);
}

} // namespace

void launch_adamw_tensors(const void *image, int64_t count, int64_t chunks, const AdamTensorConsts &k,
                          uint64_t seed, uint64_t step, hipStream_t st)
{
    StepArgs a;
    a.tensors = static_cast<const TensorEntry *>(image);
    const int32_t *chunk_tensor = reinterpret_cast<const int32_t *>(a.tensors + count);
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
    // Chunks of one launch: a grid's dimension holds fewer than 2^32 threads.
    constexpr int64_t kLaunchChunks = (int64_t)1 << 23;
    for (int64_t c = 0; c < chunks; c += kLaunchChunks) {
        const dim3 grid((unsigned)(chunks - c < kLaunchChunks ? chunks - c : kLaunchChunks));
        a.chunk_tensor = chunk_tensor + c;
        if (c == 0)
            hipLaunchKernelGGL(adamw_tensors_kernel, grid, dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL(adamw_tensors_from_kernel, grid, dim3(256), 0, st, a, (uint32_t)c);
    }
}

} // namespace qlin
