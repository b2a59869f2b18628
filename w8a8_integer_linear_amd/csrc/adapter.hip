// Low-rank adapters of many requests beside one shared INT8 projection.
//
// Token m has the adapter l = ids[m] (none if that is outside [0, L)); its
// matrices A[l] [R, K] and B[l] [N, R] and a factor scale[l].  The adapters
// read the projection's own INT8 input, x^ = sx q, in the basis of the codes
// (rotated where the projection's weight is), so a layer keeps one copy of
// its input, of one byte per element, for the projection and the adapters.
//
//   u = scale (x^ A^T)      y  = sx sw acc + bias + u B^T
//   v = scale (dY B)        dx = rotate(sg acc + v A)
//   dA[l] = sum over l's tokens of v^T x^     dB[l] = the same of dY^T u
//
// The products run on v_mfma_f32_16x16x32_bf16 with fp32 sums.  INT8 codes
// are exact in bf16; an fp32 operand is split into three bf16 terms, which hold
// its 24 bits, and a product of two such operands keeps the six partial
// products above 2^-24.  (Two terms and three products were 2.5 to 5 times as
// far from the 64-bit result as fp32 products are.)  Every lane of an
// accumulator belongs to one token, so the rows of a 16-token block that have
// another adapter are dropped by a select and never meet its matrices' values (a
// NaN in one adapter stays with its tokens).
#include <type_traits>

#include "adapter_frag.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "lowp.hpp"

namespace qlin {

namespace {

// ------------------------------------------------------------------ shrink

struct ShrinkArgs {
    const void *x;          // [M, C]
    const float *xs;        // [M] row scales of INT8 codes, or null
    const void *w;          // [L, R, C]
    const float *scale;     // [L]
    const int32_t *ids;
    int64_t M, C;
    int L, R;
    float *out;             // [M, R]
    uint16_t *terms;        // out as bf16 terms for a q of form qt
    int qt;
    // The contraction in `splits` workgroups per 32 tokens and group of ranks:
    // their sums (part: 512 RB values each) and arrival counters (zero before and
    // after).
    int splits;
    float *part;
    unsigned *count;
};

// Four values of a row of out, from rank r.
__device__ __forceinline__ void put_out(const ShrinkArgs &a, int64_t m, int r, f32x4 v)
{
    *reinterpret_cast<f32x4 *>(a.out + m * a.R + r) = v;
    const float f[4] = {v[0], v[1], v[2], v[3]};
    put_terms<4>(a.terms, a.qt, a.R, m, r, f);
}

// W of a shrink product: X_BF16 or X_F32, [L, R, C], or three bf16 terms, one
// plane [L, R, C] after another.
enum { W_TERMS = 3 };
constexpr int terms_of_w(int w) { return w == X_BF16 ? 1 : 3; }

// A 16-token operand's bytes in LDS: rows of kRowBytes, whose 16-byte chunk c
// lies at position c ^ (row & 7), so that the 16 rows that a fragment read
// takes together fall on all banks.  Rows come straight from global memory by
// buffer loads, 1 KiB per wave instruction: chunk for chunk in memory order but
// for that exchange, which stays within 128 bytes.
typedef __attribute__((address_space(3))) int8_t lds_byte;

template <int ROW_BYTES> struct RowTile {
    static constexpr int kRowBytes = ROW_BYTES, kChunks = ROW_BYTES / 16;

    // Instruction n (of rows * ROW_BYTES / 1024): the lane's row and byte.
    __device__ static __forceinline__ void slot(int n, int &row, int &byte)
    {
        const int s = n * 64 + __lane_id();
        row = s / kChunks;
        byte = 16 * ((s % kChunks) ^ (row & 7));
    }
    __device__ static __forceinline__ i32x4 read(const lds_byte *tile, int row, int byte)
    {
        typedef const __attribute__((address_space(3))) i32x4 lds_i32x4;
        return *reinterpret_cast<lds_i32x4 *>(tile + row * ROW_BYTES + 16 * ((byte / 16) ^ (row & 7)));
    }
    // Eight bytes.
    __device__ static __forceinline__ i32x2 read8(const lds_byte *tile, int row, int byte)
    {
        typedef const __attribute__((address_space(3))) i32x2 lds_i32x2;
        return *reinterpret_cast<lds_i32x2 *>(tile + row * ROW_BYTES + 16 * ((byte / 16) ^ (row & 7)) +
                                              byte % 16);
    }
};

constexpr uint32_t kPastEnd = 0x7FFFFFF0u;      // beyond every buffer below: reads zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)kPastEnd, kRsrcWord3);
}

// out[m, r] = scale xs[m] sum_c x[m, c] w[id, r, c] for 32 tokens and RB blocks of
// 16 ranks per workgroup.  512 bytes of every token's row and w's values for
// them are brought into LDS at a time, STAGES - 1 such stages ahead.  The waves
// share a stage's steps of 32 contraction indexes, an eighth each for both token
// blocks, so that w is split into terms once (fp32 x: four steps, a quarter each
// for one token block), and their sums are added at the end.  What bounds it is
// the read of x.  (Fragments straight from global memory took two to three times
// as long: neighbouring lanes hold different rows, and each was a cache access of
// its own.)  12000 tokens of 7168 bf16 values, rank 16: 34-37 us, 4.6-5.1 TB/s.
// Few tokens: the contraction is split over workgroups until there are two per
// compute unit (611 tokens, 4096 codes, rank 32 in fp32: 11 us, latency).
template <int X, int W, int RB, int STAGES>
__global__ __launch_bounds__(512) void adapter_shrink_kernel(ShrinkArgs a)
{
    constexpr int kSize = X == X_I8 ? 1 : X == X_BF16 ? 2 : 4;
    constexpr int kStep = 512 / kSize;                  // contraction indexes of a stage
    constexpr int kPlanes = W == W_TERMS ? 3 : 1, kWSize = W == X_F32 ? 4 : 2;
    using XTile = RowTile<512>;
    using WTile = RowTile<kStep * kWSize>;
    constexpr int kXBytes = 32 * 512, kWBytes = 16 * RB * kPlanes * WTile::kRowBytes;
    constexpr int kStageBytes = kXBytes + kWBytes;
    constexpr int kXLoads = kXBytes / 1024 / 8, kWLoads = (kWBytes / 1024 + 7) / 8;
    constexpr int kLoads = kXLoads + kWLoads;           // per wave and stage
    constexpr int kBlocks = X == X_F32 ? 1 : 2;         // token blocks of a wave
    constexpr int kParts = 4 * kBlocks;                 // waves per token block
    static_assert(RB * 2 * kParts * kWave * 16 <= STAGES * kStageBytes, "the sums reuse the stages");
    __shared__ __attribute__((aligned(1024))) int8_t smem[STAGES * kStageBytes];
    const int lane = __lane_id(), w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int tb0 = kBlocks == 2 ? 0 : w % 2, part = kBlocks == 2 ? w : w / 2;
    const int rb0 = blockIdx.y * RB * 16;
    const int64_t m0 = (int64_t)blockIdx.x * 32;
    const int64_t plane = (int64_t)a.L * a.R * a.C * 2;
    const int row_bytes = (int)(a.C * kSize);
    const __amdgpu_buffer_rsrc_t xr = buffer_of(static_cast<const int8_t *>(a.x) + m0 * row_bytes);
    // This workgroup's stages of the contraction.
    const int all = (int)((a.C + kStep - 1) / kStep);
    const int first = all * (int)blockIdx.z / a.splits;
    const int steps = all * ((int)blockIdx.z + 1) / a.splits - first;
    // The work is one sequence: the stages of each adapter among the tokens, one
    // adapter after another.  A cursor walks it: one where loads are issued, one
    // where they are used.  (cur < 0: past the end.)
    int id[2];
#pragma unroll
    for (int t = 0; t < 2; t++)
        id[t] = id_of(a.ids, m0 + 16 * t + lane % 16, a.M, a.L);
    struct Cursor {
        int left[2], cur, st;
        __device__ __forceinline__ void next_adapter()
        {
            cur = -1;
            st = 0;
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const uint64_t any = __ballot(left[t] >= 0);
                if (any)
                    cur = __builtin_amdgcn_readlane(left[t], (int)__builtin_ctzll(any));
            }
#pragma unroll
            for (int t = 0; t < 2; t++)
                left[t] = left[t] == cur ? -1 : left[t];
        }
        __device__ __forceinline__ void advance(int steps)
        {
            if (++st == steps)
                next_adapter();
        }
    };
    Cursor to = {{id[0], id[1]}, -1, 0};
    to.next_adapter();
    Cursor at = to;
    f32x4 acc[kBlocks][RB];
#pragma unroll
    for (int t = 0; t < kBlocks; t++)
#pragma unroll
        for (int b = 0; b < RB; b++)
            acc[t][b] = f32x4{0, 0, 0, 0};
    const bool none = at.cur < 0;
    // (Stages past the end read zeros, so that every iteration waits for the same
    // number of loads.)
    auto issue = [&](int slot) {
        lds_byte *dst = (lds_byte *)smem + slot * kStageBytes;
        const int64_t k0 = (int64_t)(to.cur >= 0 ? first + to.st : all) * kStep;
        const int64_t w0 = ((int64_t)(to.cur >= 0 ? to.cur : 0) * a.R + rb0) * a.C * kWSize;
#pragma unroll
        for (int n = 0; n < kXLoads; n++) {
            int r, byte;
            XTile::slot(w * kXLoads + n, r, byte);
            const bool ok = m0 + r < a.M && k0 * kSize + byte < row_bytes;
            const uint32_t off = ok ? (uint32_t)(r * row_bytes + byte + k0 * kSize) : kPastEnd;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                xr, (__attribute__((address_space(3))) void *)(dst + (w * kXLoads + n) * 1024), 16, off,
                0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < kWLoads; n++) {
            const int at = w * kWLoads + n;         // KiB of the stage's w
            constexpr int kKiB = kWBytes / 1024, kPlaneKiB = kKiB / kPlanes;
            // (A wave without a piece of its own repeats the last one.)
            const int piece = at < kKiB ? at : kKiB - 1, p = piece / kPlaneKiB;
            const __amdgpu_buffer_rsrc_t wr = buffer_of(static_cast<const int8_t *>(a.w) + w0 + p * plane);
            int r, byte;
            WTile::slot(piece % kPlaneKiB, r, byte);
            const int64_t in = k0 * kWSize + byte;
            const bool ok = rb0 + r < a.R && in < a.C * kWSize;
            const uint32_t off = ok ? (uint32_t)(r * a.C * kWSize + in) : kPastEnd;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                wr, (__attribute__((address_space(3))) void *)(dst + kXBytes + piece * 1024), 16, off, 0,
                0, 0);
        }
        to.advance(steps);
    };
    f32x4 s[kBlocks][RB];
#pragma unroll
    for (int t = 0; t < kBlocks; t++)
#pragma unroll
        for (int b = 0; b < RB; b++)
            s[t][b] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int st = 0; st < STAGES - 1; st++)
        issue(st);
    int slot = 0;
    while (at.cur >= 0) {
        issue(slot + STAGES - 1 < STAGES ? slot + STAGES - 1 : slot - 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads *(STAGES - 1)) : "memory");
        asm volatile("s_barrier" ::: "memory");
        const lds_byte *xt = (const lds_byte *)smem + slot * kStageBytes;
        const lds_byte *wt = xt + kXBytes;
        constexpr int kMine = kStep / 32 / kParts;      // steps of this wave
#pragma unroll
        for (int q = 0; q < kMine; q++) {
            const int k = (part * kMine + q) * 32 + 8 * (lane / 16);
            Frag<terms_of(X)> xf[kBlocks];
#pragma unroll
            for (int t = 0; t < kBlocks; t++) {
                const int row = (tb0 + t) * 16 + lane % 16;
                if constexpr (X == X_BF16) {
                    xf[t].t[0] = __builtin_bit_cast(bf16x8, XTile::read(xt, row, 2 * k));
                } else if constexpr (X == X_I8) {
                    float v[8];
                    codes_to_float(XTile::read8(xt, row, k), v);
                    xf[t].t[0] = round8(v);
                } else {
                    float v[8];
                    unpack8<false>({__builtin_bit_cast(f32x4, XTile::read(xt, row, 4 * k)),
                                    __builtin_bit_cast(f32x4, XTile::read(xt, row, 4 * k + 16))},
                                   v);
                    xf[t] = split8(v);
                }
            }
#pragma unroll
            for (int b = 0; b < RB; b++) {
                Frag<terms_of_w(W)> wf;
                const int r = 16 * b + lane % 16;
                if constexpr (W == X_F32) {
                    float v[8];
                    unpack8<false>({__builtin_bit_cast(f32x4, WTile::read(wt, r, 4 * k)),
                                    __builtin_bit_cast(f32x4, WTile::read(wt, r, 4 * k + 16))},
                                   v);
                    wf = split8(v);
                } else {
#pragma unroll
                    for (int p = 0; p < kPlanes; p++)
                        wf.t[p] = __builtin_bit_cast(
                            bf16x8, WTile::read(wt + p * (kWBytes / kPlanes), r, 2 * k));
                }
#pragma unroll
                for (int t = 0; t < kBlocks; t++)
                    s[t][b] = mfma(wf, xf[t], s[t][b]);
            }
        }
        if (at.st == steps - 1) {
#pragma unroll
            for (int t = 0; t < kBlocks; t++)
#pragma unroll
                for (int b = 0; b < RB; b++) {
                    acc[t][b] = (kBlocks == 2 ? id[t] : tb0 ? id[1] : id[0]) == at.cur ? s[t][b] : acc[t][b];
                    s[t][b] = f32x4{0, 0, 0, 0};
                }
        }
        // Every wave has read the stage before the next issue refills it.
        lds_barrier();
        at.advance(steps);
        slot = slot + 1 < STAGES ? slot + 1 : 0;
    }
    // (The stages past the end are still landing.)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
    // (Without any adapter the first split writes the zeros.)
    if (none && blockIdx.z > 0)
        return;
    f32x4 *red = reinterpret_cast<f32x4 *>(smem);       // [RB][2][kParts][64]
#pragma unroll
    for (int t = 0; t < kBlocks; t++)
#pragma unroll
        for (int b = 0; b < RB; b++)
            red[((b * 2 + tb0 + t) * kParts + part) * kWave + lane] = acc[t][b];
    __syncthreads();
    // Waves 0 .. 2 RB - 1: token block tb, ranks rb.
    const int tb = w % 2, rb = w / 2;
    const int mine_id = tb ? id[1] : id[0];
    const int64_t m = m0 + 16 * tb + lane % 16;
    const int r = rb0 + 16 * rb + 4 * (lane / 16);
    f32x4 sum = {0, 0, 0, 0};
    if (rb < RB) {
        sum = red[(w * kParts) * kWave + lane];
#pragma unroll
        for (int q = 1; q < kParts; q++)
            sum += red[(w * kParts + q) * kWave + lane];
    }
    if (!none && a.splits > 1) {
        // The sums cross XCDs, whose L2s are not coherent: stored and read with
        // the device-scope bit, the stores complete before the arrival counts.
        constexpr int kCoherentBit = 16;
        const int unit = blockIdx.x * gridDim.y + blockIdx.y;
        const __amdgpu_buffer_rsrc_t pr =
            buffer_of(a.part + (int64_t)unit * a.splits * (RB * 2 * kWave * 4));
        const uint32_t mine = (w * kWave + lane) * 16;
        constexpr uint32_t kPart = RB * 2 * kWave * 16;
        if (rb < RB)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, sum), pr,
                                                   blockIdx.z * kPart + mine, 0, kCoherentBit);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        int *flag = reinterpret_cast<int *>(smem);
        if (threadIdx.x == 0) {
            const unsigned arrived = atomicAdd(a.count + unit, 1u);
            *flag = arrived == (unsigned)(a.splits - 1);
            if (*flag)
                atomicExch(a.count + unit, 0u);
        }
        __syncthreads();
        if (!*flag || rb >= RB)
            return;
        // In the order of the splits, four loads in flight.
        sum = f32x4{0, 0, 0, 0};
        for (int z0 = 0; z0 < a.splits; z0 += 4) {
            f32x4 v[4];
#pragma unroll
            for (int z = 0; z < 4; z++)
                v[z] = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               pr, z0 + z < a.splits ? (z0 + z) * kPart + mine : kPastEnd, 0, kCoherentBit));
#pragma unroll
            for (int z = 0; z < 4; z++)
                sum += v[z];
        }
    }
    if (rb < RB && m < a.M && r < a.R) {
        const float f = mine_id >= 0 ? a.scale[mine_id] * (a.xs ? a.xs[m] : 1.0f) : 0.0f;
        put_out(a, m, r, mine_id >= 0 ? sum * f : f32x4{0, 0, 0, 0});
    }
}

// Tokens of the weight-streaming product, which does not read the terms.
constexpr int64_t kSkinnyTokens = 16;

// The same for a few tokens: one wave per token and rank, whose read of w (the
// ranks of one token's adapter in as many waves) is what takes the time (7 tokens,
// 4096 codes, rank 16: 3.5 us).
template <int W> __global__ __launch_bounds__(256) void adapter_shrink_few_kernel(ShrinkArgs a)
{
    const int lane = __lane_id();
    const int64_t at = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
    const int64_t m = at / a.R;
    const int r = (int)(at % a.R);      // (R is a multiple of 4: one token per workgroup)
    const int id = id_of(a.ids, m, a.M, a.L);
    float s = 0.0f;
    if (id >= 0) {
        const int64_t x0 = m * a.C, w0 = ((int64_t)id * a.R + r) * a.C;
        // Four pieces of 1024 contraction indexes are loaded at once; those past
        // the end read the last values and do not count.
        constexpr int kAtOnce = 4;
        constexpr bool kBf = W == X_BF16;
        for (int64_t k0 = lane * 16; k0 < a.C; k0 += kAtOnce * kWave * 16) {
            i32x4 q[kAtOnce];
            Raw8<kBf> wr[kAtOnce][2];
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                const int64_t k = k0 + i * kWave * 16 < a.C ? k0 + i * kWave * 16 : a.C - 16;
                q[i] = *reinterpret_cast<const i32x4 *>(static_cast<const int8_t *>(a.x) + x0 + k);
                wr[i][0] = load_raw8<kBf>(a.w, w0 + k);
                wr[i][1] = load_raw8<kBf>(a.w, w0 + k + 8);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                float x[16], w[16], t = 0.0f;
                codes_to_float(i32x2{q[i][0], q[i][1]}, x);
                codes_to_float(i32x2{q[i][2], q[i][3]}, x + 8);
                unpack8<kBf>(wr[i][0], w);
                unpack8<kBf>(wr[i][1], w + 8);
#pragma unroll
                for (int e = 0; e < 16; e++)
                    t = __builtin_fmaf(x[e], w[e], t);
                s = k0 + i * kWave * 16 < a.C ? s + t : s;
            }
        }
    }
    s = wave_all(s, [](float p, float q) { return p + q; });
    if (lane == 0) {
        const float v = id >= 0 ? s * (a.scale[id] * (a.xs ? a.xs[m] : 1.0f)) : 0.0f;
        a.out[m * a.R + r] = v;
        if (a.M > kSkinnyTokens) {
            const float f[1] = {v};
            put_terms<1>(a.terms, a.qt, a.R, m, r, f);
        }
    }
}

// Most waves (tokens times ranks) of the kernel above, which reads an adapter once
// per token, but all adapters at once.  us for the call, 4096 -> 4096 in bf16, this
// kernel / the tiles of 32 tokens:
//                                        1024      4096      8192     16384
//   rank 16, nine requests in a row      39/47     40/42     45/44     59/53
//   rank 64, nine requests in a row      63/75     49/55     48/49     53/48
//   rank 16, 8 adapters in any order     45/58     48/58     54/62     73/77
//   rank 16, 256 adapters in any order   56/102    61/101    70/108    97/128
// (The host knows neither the number of distinct adapters nor their order: the bound
// is where no case loses, and mixed tokens above it pay up to half as much again.)
constexpr int64_t kFewWaves = 4096;

// Workgroups that a product of fewer units (32 tokens by a group of ranks) than
// compute units is split up to, fewest stages of a split's, and most units that
// are split at all: each has an arrival counter.
constexpr int kCus = 256, kSplitGroups = 2 * kCus, kSplitStages = 2, kMaxUnits = 2 * kCus;
static_assert(kMaxUnits * 4 <= kAdapterCountBytes, "arrival counters");
constexpr size_t kPartBytes = (size_t)2 * kMaxUnits * 2 * 512 * 4;

// Splits of a product of `units` workgroups and `stages` stages each.  More units
// than compute units are halved where that takes half a round less (375 units of
// 7168 bf16 values: 43 us in one piece, 37 us in two).
int splits_of(int64_t units, int64_t stages)
{
    if (units > kMaxUnits)
        return 1;
    auto rounds = [](int64_t n) { return (n + kCus - 1) / kCus; };
    int64_t n = units <= kCus ? kSplitGroups / units : rounds(2 * units) < 2 * rounds(units) ? 2 : 1;
    n = n < stages / kSplitStages ? n : stages / kSplitStages;
    return (int)(n < 1 ? 1 : n);
}

template <int X, int W, int RB> void go_shrink(ShrinkArgs a, hipStream_t st)
{
    constexpr int kSize = X == X_I8 ? 1 : X == X_BF16 ? 2 : 4;
    constexpr int kStage = 32 * 512 + 16 * RB * (W == W_TERMS ? 3 : 1) * (W == X_F32 ? 4 : 2) * 512 / kSize;
    constexpr int kStages = kStage <= 26 * 1024 ? 3 : 2;
    const int64_t blocks = (a.M + 31) / 32, groups = (a.R + 16 * RB - 1) / (16 * RB);
    a.splits = splits_of(blocks * groups, (a.C * kSize + 511) / 512);
    const dim3 grid((unsigned)blocks, (unsigned)groups, (unsigned)a.splits);
    hipLaunchKernelGGL((adapter_shrink_kernel<X, W, RB, kStages>), grid, dim3(512), 0, st, a);
}

template <int X, int W> void run_shrink(const ShrinkArgs &a, hipStream_t st)
{
    if constexpr (X == X_I8) {
        if (a.M * a.R <= kFewWaves) {
            hipLaunchKernelGGL(adapter_shrink_few_kernel<W>, dim3((unsigned)(a.M * a.R / 4)), dim3(256), 0,
                               st, a);
            return;
        }
    }
    // 32 ranks share x's stage where w's fits beside it and two workgroups per
    // compute unit are left (5376 codes, bf16, a product of 16 columns: 12000
    // tokens of rank 64, 80 us for the call against 89 us; 4200 of rank 64, 62 us
    // against 60 us; 12000 of rank 32, 68 us against 67 us).
    if constexpr (W == X_BF16) {
        if ((a.M + 31) / 32 * ((a.R + 31) / 32) >= 2 * kCus)
            return go_shrink<X, W, 2>(a, st);
    }
    go_shrink<X, W, 1>(a, st);
}

// ------------------------------------------------------------------ expand

// out[m, c] += sum_r p[m, r] q[id, c, r], for products of so few tiles that
// adding the term in their epilogues would leave it to a few compute units: block
// (bx, by) has 16 tokens by 256 columns, 64 per wave.  QT: q as one bf16 term (1),
// as three (4), or fp32 (0).  DX: the sums go through LDS (kExpandTile floats) and
// are rotated in blocks along their rows before they are written (the rotation of
// dX, which the product's own epilogue cannot do before the term is added; a
// launch of its own cost 5 us of 107 at 333 tokens, 4096 x 4096, rank 64 in fp32).
// Reading q bounds it: three terms took 8 us there, their six pairs 13 us.
// A row's pitch keeps the four column groups of a write on banks of their own.
constexpr int kExpandPitch = 256 + 4, kExpandTile = 16 * kExpandPitch;

template <int QT, bool DX>
__device__ __forceinline__ void expand(const AdapterTermArgs &a, int64_t bx, int64_t by, float *tile)
{
    const int lane = __lane_id(), w = threadIdx.x / kWave, R = a.ad.R;
    const int64_t m = by * 16 + lane % 16;
    const int64_t c0 = bx * 256 + w * 64;
    const int id = id_of(a.ad.ids, m, a.M, a.ad.L);
    f32x4 acc[4];
#pragma unroll
    for (int b = 0; b < 4; b++) {
        const int64_t c = c0 + 16 * b + 4 * (lane / 16);
        acc[b] = f32x4{0, 0, 0, 0};
        if ((DX ? m < a.M : id >= 0) && c < a.C)
            acc[b] = *reinterpret_cast<const f32x4 *>(a.out + m * a.C + c);
    }
    constexpr int kTerms = QT == 1 ? 1 : 3;
    const int length = (QT == 1 ? 3 : 1) * R, steps = terms_steps(QT, R);
    struct Step {
        Frag<kTerms> p, q[4];
    };
    for_adapters(id, [&](int cur, bool mine) {
        auto load = [&](int k0) {
            const int k = k0 + 8 * (lane / 16);
            const bool ok = k < length;
            const int r = QT == 1 ? k - ((k >= R) + (k >= 2 * R)) * R : k;
            Step f;
#pragma unroll
            for (int t = 0; t < kTerms; t++)
                f.p.t[t] = load_frag<X_BF16>(
                    a.ad.terms, ((by * steps + k0 / 32 * kTerms + t) * 64 + lane) * 8, ok).t[0];
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const int64_t c = c0 + 16 * b + lane % 16;
                if constexpr (QT == 4) {
                    const int64_t block = (int64_t)cur * (a.C / 16) + c / 16;
#pragma unroll
                    for (int t = 0; t < kTerms; t++)
                        f.q[b].t[t] = load_frag<X_BF16>(
                            a.ad.q, (block * steps + k0 / 32 * kTerms + t) * 512 + lane * 8, ok && c < a.C).t[0];
                } else
                    f.q[b] = load_frag<QT == 0 ? X_F32 : X_BF16>(
                        a.ad.q, ((int64_t)cur * a.C + c) * R + r, ok && c < a.C);
            }
            return f;
        };
        auto use = [&](const Step &f) {
#pragma unroll
            for (int b = 0; b < 4; b++) {
                const f32x4 t = mfma(f.q[b], f.p, acc[b]);
                acc[b] = mine ? t : acc[b];
            }
        };
        // Several steps at a time, so that their loads are in flight together (those
        // past the end are zeros).
        constexpr int kAtOnce = QT == 1 ? 4 : 2;
        for (int k0 = 0; k0 < length; k0 += 32 * kAtOnce) {
            Step f[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; i++)
                f[i] = load(k0 + 32 * i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kAtOnce; i++)
                use(f[i]);
        }
    });
    if constexpr (DX) {
#pragma unroll
        for (int b = 0; b < 4; b++)
            *reinterpret_cast<f32x4 *>(tile + (lane % 16) * kExpandPitch + w * 64 + 16 * b + 4 * (lane / 16)) =
                acc[b];
        __syncthreads();
        // Eight consecutive values per lane, 32 lanes per row.  (All lanes take
        // part in the exchange; blocks lie inside a row's C columns or outside.)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int chunk = i * 256 + threadIdx.x, row = chunk / 32, col = chunk % 32 * 8;
            float v[8];
            load8<false>(tile, row * kExpandPitch + col, v);
            if (a.had)
                fwht8_lanes(v, a.had, a.cb);
            const int64_t om = by * 16 + row, oc = bx * 256 + col;
            if (om < a.M && oc < a.C)
                store8(a.out, om * a.C + oc, v);
        }
    } else {
        if (id < 0)
            return;
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const int64_t c = c0 + 16 * b + 4 * (lane / 16);
            if (c < a.C)
                *reinterpret_cast<f32x4 *>(a.out + m * a.C + c) = acc[b];
        }
    }
}

template <int QT> __global__ __launch_bounds__(256) void adapter_expand_kernel(AdapterTermArgs a)
{
    expand<QT, false>(a, blockIdx.x, blockIdx.y, nullptr);
}

// ------------------------------------------------------- grouping of tokens

// A stable counting sort of the tokens by adapter, in one workgroup: each of 16
// waves counts its own run of tokens, the counts become first places (adapter
// by adapter, and for one adapter wave by wave), and each wave places its
// tokens 64 at a time, one adapter among them after another.  Tokens without
// an adapter come last.  The reads' latency is what takes the time: a wave
// loads 512 tokens' adapters at once.
constexpr int kGroupWaves = 16;

__global__ __launch_bounds__(kGroupWaves *kWave) void adapter_group_kernel(const int32_t *__restrict__ ids,
                                                                           int64_t M, int L,
                                                                           int32_t *__restrict__ order,
                                                                           int32_t *__restrict__ start)
{
    __shared__ int count[kGroupWaves][kMaxAdapters + 1];
    __shared__ int total[kMaxAdapters + 1];
    const int bins = L + 1, t = threadIdx.x, w = t / kWave, lane = __lane_id();
    for (int i = t; i < kGroupWaves * bins; i += kGroupWaves * kWave)
        count[i / bins][i % bins] = 0;
    __syncthreads();
    const int64_t per = ((M + kGroupWaves * kWave - 1) / (kGroupWaves * kWave)) * kWave;
    const int64_t r0 = w * per < M ? w * per : M, r1 = r0 + per < M ? r0 + per : M;
    // f(m, bin, mask, n) for each adapter among 64 tokens of the wave's run; of
    // 768 tokens with one adapter f is called at once, with a full mask and n =
    // 12 groups of 64.  (The groups go through LDS so that the loop over them
    // stays rolled: fetching unrolled code once costs more than running it.)
    constexpr int kAtOnce = 12;
    __shared__ int16_t seen[kGroupWaves][kAtOnce * kWave];
    auto for_runs = [&](auto f) {
        for (int64_t m0 = r0; m0 < r1; m0 += kAtOnce * kWave) {
            int b[kAtOnce];
            bool same = true;
#pragma unroll
            for (int q = 0; q < kAtOnce; q++) {
                const int64_t m = m0 + q * kWave + lane;
                b[q] = ids[m < r1 ? m : r1 - 1];
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < kAtOnce; q++) {
                const int64_t m = m0 + q * kWave + lane;
                b[q] = m >= r1 ? -1 : b[q] >= 0 && b[q] < L ? b[q] : L;
                seen[w][q * kWave + lane] = (int16_t)b[q];
                same = same && b[q] == __builtin_amdgcn_readfirstlane(b[0]);
            }
            if (__all(same)) {
                f(m0 + lane, __builtin_amdgcn_readfirstlane(b[0]), ~0ull, kAtOnce);
                continue;
            }
#pragma unroll 1
            for (int q = 0; q < kAtOnce && m0 + q * kWave < r1; q++) {
                const int bin = seen[w][q * kWave + lane];
                uint64_t left = __ballot(bin >= 0);
                while (left) {
                    const int cur = __builtin_amdgcn_readlane(bin, (int)__builtin_ctzll(left));
                    const uint64_t mask = __ballot(bin == cur);
                    f(m0 + q * kWave + lane, cur, mask, 1);
                    left &= ~mask;
                }
            }
        }
    };
    for_runs([&](int64_t, int bin, uint64_t mask, int n) {
        if (lane == 0)
            count[w][bin] += n * __popcll(mask);
    });
    __syncthreads();
    for (int b = t; b < bins; b += kGroupWaves * kWave) {
        int s = 0;
        for (int i = 0; i < kGroupWaves; i++)
            s += count[i][b];
        total[b] = s;
    }
    __syncthreads();
    if (w == 0) {       // exclusive prefix sums of the totals, 64 bins at a time
        int before = 0;
        for (int b0 = 0; b0 < bins; b0 += kWave) {
            const int v = b0 + lane < bins ? total[b0 + lane] : 0;
            int s = v;
            for (int o = 1; o < kWave; o <<= 1) {
                const int x = __shfl_up(s, o);
                s += lane >= o ? x : 0;
            }
            if (b0 + lane < bins)
                total[b0 + lane] = before + s - v;
            before += __shfl(s, kWave - 1);
        }
    }
    __syncthreads();
    for (int b = t; b < bins; b += kGroupWaves * kWave) {
        int s = total[b];
        start[b] = s;       // start[L]: the first token without an adapter
        for (int i = 0; i < kGroupWaves; i++) {
            const int c = count[i][b];
            count[i][b] = s;
            s += c;
        }
    }
    __syncthreads();
    for_runs([&](int64_t m, int bin, uint64_t mask, int n) {
        const int first = count[w][bin];
        const int at = first + __popcll(mask & ((1ull << lane) - 1));
        for (int q = 0; q < n; q++)
            if ((mask >> lane) & 1)
                order[at + q * kWave] = (int32_t)m + q * kWave;
        if (lane == 0)
            count[w][bin] = first + n * __popcll(mask);
    });
}

// ------------------------------------------------------- adapter gradients

// The tokens of an adapter are split into slabs of kSlab; a table entry says
// which adapter a slab has and where its tokens lie in the grouped order.
constexpr int kSlab = 256;

struct Slab {
    int32_t adapter, first, rows, pad;
};

struct PrepArgs {
    const void *a, *b;      // [L, R, K], [L, N, R]
    uint16_t *at, *bt;
    int64_t N, K, M;
    int L, R, qt, slabs;    // qt: the form of A's terms
    const int32_t *start;
    Slab *table;            // [slabs]
    int32_t *first;         // [L + 1]: the first slab of each adapter
    // Where the gradients are finished by their own kernel: cleared for adapters
    // without tokens, and its arrival counters; else null.
    float *da, *db;
    unsigned *count;
    int64_t counts;
};

// Adapter l's tokens in the grouped order, as one slab, within the M tokens that
// there are whatever start holds.
__device__ __forceinline__ Slab tokens_of(const PrepArgs &p, int l)
{
    int64_t s0 = p.start[l], s1 = p.start[l + 1];
    s0 = s0 < 0 ? 0 : s0 > p.M ? p.M : s0;
    s1 = s1 < s0 ? s0 : s1 > p.M ? p.M : s1;
    return Slab{l, (int32_t)s0, (int32_t)(s1 - s0), 0};
}

// One 32 x 32 tile of src [rows, cols], turned: put(c, r, bits or value) for
// element (r, c), with neighbouring lanes at neighbouring r.
template <bool WB, typename F>
__device__ __forceinline__ void transpose_tile(const void *src, int64_t s0, int64_t rows, int64_t cols,
                                               int64_t r0, int64_t c0, F put)
{
    __shared__ uint32_t tile[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
#pragma unroll
    for (int i = y; i < 32; i += 8)
        if (r0 + i < rows && c0 + x < cols) {
            const int64_t at = s0 + (r0 + i) * cols + c0 + x;
            if constexpr (WB)
                tile[i][x] = static_cast<const uint16_t *>(src)[at];
            else
                tile[i][x] = static_cast<const uint32_t *>(src)[at];
        }
    __syncthreads();
#pragma unroll
    for (int i = y; i < 32; i += 8)
        if (c0 + i < cols && r0 + x < rows)
            put(c0 + i, r0 + x, tile[x][i]);
}

// What the backward kernels need first, in one launch: B transposed for the
// product with dY, A for dX's epilogue (both then have the contraction index
// contiguous), fp32 ones split into bf16 terms (B [3, L, R, N]; A, per adapter, in
// the layout of adapter_frag.hpp, a row per column),
// the table of slabs, and zeros in the arrival counters and in the gradients of
// adapters without tokens.  Workgroup 0 of adapter 0 makes the table, 256 adapters
// at a time.
template <bool WB> __global__ __launch_bounds__(256) void adapter_prep_kernel(PrepArgs p)
{
    const int t = threadIdx.x;
    if (blockIdx.x > 0) {
        const int64_t rt = (p.R + 31) / 32, nt = (p.N + 31) / 32, l = blockIdx.y;
        const int64_t k = blockIdx.x - 1;
        const int64_t sb = l * p.N * p.R, sa = l * p.K * p.R;
        if (p.da && tokens_of(p, (int)l).rows == 0) {
            // (As many elements per workgroup as a tile of 32 x 32 has.)
            const bool is_b = k < rt * nt;
            const int64_t size = (is_b ? p.N : p.K) * p.R, i0 = (is_b ? k : k - rt * nt) * 1024;
            for (int64_t i = i0 + t; i < i0 + 1024 && i < size; i += 256)
                (is_b ? p.db + sb : p.da + sa)[i] = 0.0f;
            return;
        }
        if (k < rt * nt) {
            const int64_t plane = (int64_t)p.L * p.R * p.N;
            transpose_tile<WB>(p.b, sb, p.N, p.R, k / rt * 32, k % rt * 32,
                               [&](int64_t r, int64_t n, uint32_t bits) {
                                   uint16_t *to = p.bt + sb + r * p.N + n;
                                   if constexpr (WB) {
                                       *to = (uint16_t)bits;
                                   } else {
                                       float v = __uint_as_float(bits);
#pragma unroll
                                       for (int q = 0; q < 3; q++) {
                                           const uint32_t w = pack_bf16x2(v, 0.0f);
                                           to[q * plane] = (uint16_t)w;
                                           v = v - bf16_lo(w);
                                       }
                                   }
                               });
        } else {
            const int64_t r0 = (k - rt * nt) % rt * 32, c0 = (k - rt * nt) / rt * 32;
            if constexpr (WB) {
                transpose_tile<WB>(p.a, sa, p.R, p.K, r0, c0, [&](int64_t c, int64_t r, uint32_t bits) {
                    p.at[sa + c * p.R + r] = (uint16_t)bits;
                });
            } else if (t < 128) {
                // Eight ranks of a column per thread (the reads are coalesced
                // over the columns).
                const int64_t c = c0 + t % 32, r = r0 + t / 32 * 8;
                if (c < p.K && r < p.R) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        v[e] = static_cast<const float *>(p.a)[sa + (r + e) * p.K + c];
                    put_other(p.at + l * (p.K / 16) * terms_steps(p.qt, p.R) * 512, p.qt, p.R, c, (int)r, v);
                }
            }
        }
        return;
    }
    if (blockIdx.y > 0)
        return;
    __shared__ int sum[4];
    const int w = t / kWave, lane = __lane_id();
    for (int i = t; i < p.slabs; i += 256)
        p.table[i] = Slab{0, 0, 0, 0};
    for (int64_t i = t; i < p.counts; i += 256)
        p.count[i] = 0;
    int base = 0;
    for (int l0 = 0; l0 <= p.L; l0 += 256) {
        __syncthreads();        // the zeros above, and the last round's sums
        const int l = l0 + t;
        const Slab mine = l < p.L ? tokens_of(p, l) : Slab{0, 0, 0, 0};
        const int n = (mine.rows + kSlab - 1) / kSlab;
        int s = n;
        for (int o = 1; o < kWave; o <<= 1) {
            const int x = __shfl_up(s, o);
            s += lane >= o ? x : 0;
        }
        if (lane == kWave - 1)
            sum[w] = s;
        __syncthreads();
        int before = base + s - n;
        for (int i = 0; i < 4; i++) {
            before += i < w ? sum[i] : 0;
            base += sum[i];
        }
        if (l <= p.L)
            p.first[l] = before < p.slabs ? before : p.slabs;
        for (int i = 0; i < n && before + i < p.slabs; i++) {
            const int past = i * kSlab, rows = mine.rows - past;
            p.table[before + i] = Slab{l, mine.first + past, rows < kSlab ? rows : kSlab, 0};
        }
    }
}

struct OuterArgs {
    const float *p;         // [M, R]
    const float *ps;        // [M] factors of p's rows, or null
    const void *x;          // [M, C]
    const int32_t *order;
    const Slab *table;
    int64_t M, C;
    int R;
    float *part;            // per slab: [R, C], or [C, R] (TRANS)
    // For few tokens, the adapters' sums over their slabs are made here too (else
    // out is null): per adapter as part per slab; first: each adapter's first
    // slab; count [L, gridDim.x]: arrivals, zero before.
    float *out;
    const int32_t *first;
    unsigned *count;
};

// Values that other workgroups, on other XCDs whose L2s are not coherent with
// this one's, read or have written.
__device__ __forceinline__ void store_shared(float *p, f32x4 v)
{
    typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
    const u64x2 w = __builtin_bit_cast(u64x2, v);
    unsigned long long *to = reinterpret_cast<unsigned long long *>(p);
    __hip_atomic_store(to, w[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(to + 1, w[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ f32x4 load_shared(float *p)
{
    typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
    unsigned long long *from = reinterpret_cast<unsigned long long *>(p);
    u64x2 w;
    w[0] = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    w[1] = __hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_bit_cast(f32x4, w);
}

// An LDS tile of 32 tokens by COLS bf16 values, rows as in memory.  The
// operands have the token index as the contraction, which the transposing read
// brings into a lane: in each 16-lane group lane s points at row s / 4, columns
// 4 (s % 4) of its block, and lane i gets the four rows of column i.  Rows are
// 32 bytes apart in the banks and every eight of them another 128, so the 64
// lanes of a read fall on all banks twice.
template <int COLS> struct TokenTile {
    static constexpr int kRow = COLS + 16;
    static constexpr int kSize = 32 * kRow + 3 * 64;
    __device__ static __forceinline__ int at(int row, int col) { return row * kRow + (row / 8) * 64 + col; }

    // Columns c0 .. c0 + 15, all 32 tokens, as an MFMA operand.
    __device__ static __forceinline__ bf16x8 operand(const uint16_t *tile, int c0)
    {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int s = __lane_id() % 16, g = __lane_id() / 16;
        s16x4 h[2];
#pragma unroll
        for (int k = 0; k < 2; k++)
            h[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(tile + at(8 * g + 4 * k + s / 4, c0 + 4 * (s % 4))));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Columns of x per workgroup: fp32 ones take six products of terms each.
constexpr int outer_cols(int x) { return x == X_F32 ? 128 : 256; }

// part[slab] = sum over the slab's tokens of p^T x, for outer_cols(X) columns, a
// quarter of them per wave.  32 tokens at a time are brought into LDS, split into bf16 terms on
// the way; the next ones' loads are in flight meanwhile.  The read of x bounds
// it: 12000 tokens of 7168 bf16 values and 5376 codes, rank 16, take 36-38 us for
// both gradients, 6.2-6.5 TB/s, part of it out of the infinity cache, since the
// product with B has just read the same dY.
template <int X, bool TRANS, int RB>
__device__ __forceinline__ void outer_product(const OuterArgs &a, int column_block, uint16_t *smem)
{
    constexpr int XT = terms_of(X), kCols = outer_cols(X), CB = kCols / 64;
    using XTile = TokenTile<kCols>;
    using PTile = TokenTile<RB * 16>;
    uint16_t(&xs)[XT][XTile::kSize] = *reinterpret_cast<uint16_t(*)[XT][XTile::kSize]>(smem);
    uint16_t(&ps)[3][PTile::kSize] =
        *reinterpret_cast<uint16_t(*)[3][PTile::kSize]>(smem + XT * XTile::kSize);
    const Slab s = a.table[blockIdx.y];
    if (s.rows <= 0)
        return;
    const int t = threadIdx.x, w = t / kWave, lane = __lane_id();
    const int64_t c0 = (int64_t)column_block * kCols;
    f32x4 acc[CB][RB];
#pragma unroll
    for (int b = 0; b < CB; b++)
#pragma unroll
        for (int r = 0; r < RB; r++)
            acc[b][r] = f32x4{0, 0, 0, 0};
    // Thread t brings an eighth of the columns of token t / 8, sixteen bytes at a
    // time (eight threads read 128 bytes in a row), and two ranks in 16 of p, into
    // one of two register sets.
    constexpr int kSets = 2;
    constexpr int kSize = X == X_I8 ? 1 : X == X_BF16 ? 2 : 4;
    constexpr int kPieces = kCols * kSize / 128, kPer = 16 / kSize;       // 16-byte pieces, values in one
    const int row = t / 8, pc = (t % 8) * 2;
    auto piece_col = [&](int q) { return (t % 8) * kPer + q * 8 * kPer; };
    auto token = [&](int i0) {
        const int i = i0 + row;
        const int64_t m = i < s.rows ? a.order[s.first + i] : -1;
        return m >= 0 && m < a.M ? m : (int64_t)-1;
    };
    i32x4 xr[kSets][kPieces];
    f32x2 pr[kSets][RB];
    float f[kSets];
    auto load = [&](int64_t m, auto S) {
        constexpr int k = decltype(S)::value;
        const bool live = m >= 0;
        const int64_t mm = live ? m : 0;
#pragma unroll
        for (int q = 0; q < kPieces; q++) {
            xr[k][q] = i32x4{0, 0, 0, 0};
            if (live && c0 + piece_col(q) < a.C)
                xr[k][q] = *reinterpret_cast<const i32x4 *>(static_cast<const char *>(a.x) +
                                                            (mm * a.C + c0 + piece_col(q)) * kSize);
        }
#pragma unroll
        for (int r = 0; r < RB; r++) {
            pr[k][r] = f32x2{0, 0};
            if (live && 16 * r + pc < a.R)
                pr[k][r] = *reinterpret_cast<const f32x2 *>(a.p + mm * a.R + 16 * r + pc);
        }
        f[k] = live && a.ps ? a.ps[mm] : 1.0f;
    };
    int64_t next = -1;
    // 32 tokens from i0, which set S holds; it is then loaded with those
    // 32 kSets tokens on.
    auto step = [&](int i0, auto S) {
        constexpr int k = decltype(S)::value;
        lds_barrier();
#pragma unroll
        for (int q = 0; q < kPieces; q++) {
            const i32x4 raw = xr[k][q];
            const int at = XTile::at(row, piece_col(q));
            if constexpr (X == X_BF16) {
                *reinterpret_cast<i32x4 *>(&xs[0][at]) = raw;
            } else if constexpr (X == X_I8) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float v[8];
                    codes_to_float(i32x2{raw[2 * h], raw[2 * h + 1]}, v);
                    *reinterpret_cast<bf16x8 *>(&xs[0][at + 8 * h]) = round8(v);
                }
            } else {
                f32x4 v = __builtin_bit_cast(f32x4, raw);
#pragma unroll
                for (int h = 0; h < 3; h++) {
                    const i32x2 b = {(int)pack_bf16x2(v[0], v[1]), (int)pack_bf16x2(v[2], v[3])};
                    *reinterpret_cast<i32x2 *>(&xs[h][at]) = b;
                    v = v - f32x4{bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])};
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RB; r++) {
            float v0 = pr[k][r][0] * f[k], v1 = pr[k][r][1] * f[k];
#pragma unroll
            for (int q = 0; q < 3; q++) {
                const uint32_t b = pack_bf16x2(v0, v1);
                *reinterpret_cast<uint32_t *>(&ps[q][PTile::at(row, 16 * r + pc)]) = b;
                v0 = v0 - bf16_lo(b);
                v1 = v1 - bf16_hi(b);
            }
        }
        // (No fence: the loads of the other set stay in flight.)
        lds_barrier();
        load(next, S);          // (zeros after the last tokens)
        next = token(i0 + 32 * (kSets + 1));
        __builtin_amdgcn_sched_barrier(0);
        Frag<XT> xf[CB];
#pragma unroll
        for (int b = 0; b < CB; b++)
#pragma unroll
            for (int q = 0; q < XT; q++)
                xf[b].t[q] = XTile::operand(xs[q], w * (kCols / 4) + 16 * b);
#pragma unroll
        for (int r = 0; r < RB; r++) {
            Frag<3> pf;
#pragma unroll
            for (int q = 0; q < 3; q++)
                pf.t[q] = PTile::operand(ps[q], 16 * r);
#pragma unroll
            for (int b = 0; b < CB; b++)
                acc[b][r] = TRANS ? mfma(pf, xf[b], acc[b][r]) : mfma(xf[b], pf, acc[b][r]);
        }
    };
    constexpr std::integral_constant<int, 0> kSet0{};
    constexpr std::integral_constant<int, 1> kSet1{};
    load(token(0), kSet0);
    load(token(32), kSet1);
    next = token(32 * kSets);
    for (int i0 = 0; i0 < s.rows; i0 += 64) {
        step(i0, kSet0);
        if (i0 + 32 < s.rows)
            step(i0 + 32, kSet1);
    }
    const int64_t size = (int64_t)a.R * a.C;
    // f(index within one gradient, value) for this lane's results.
    auto for_results = [&](auto f) {
#pragma unroll
        for (int b = 0; b < CB; b++)
#pragma unroll
            for (int rb = 0; rb < RB; rb++) {
                const int64_t cb = c0 + w * (kCols / 4) + 16 * b;
                const int64_t c = cb + (TRANS ? lane % 16 : 4 * (lane / 16));
                const int r = 16 * rb + (TRANS ? 4 * (lane / 16) : lane % 16);
                if (c < a.C && r < a.R)
                    f(TRANS ? c * a.R + r : r * a.C + c, acc[b][rb]);
            }
    };
    float *part = a.part + (int64_t)blockIdx.y * size;
    if (!a.out) {
        for_results([&](int64_t at, f32x4 v) { *reinterpret_cast<f32x4 *>(part + at) = v; });
        return;
    }
    float *out = a.out + (int64_t)s.adapter * size;
    const int k0 = a.first[s.adapter], k1 = a.first[s.adapter + 1];
    if (k1 - k0 > 1) {
        // The last of the adapter's slabs to arrive adds them up, in their order.
        for_results([&](int64_t at, f32x4 v) { store_shared(part + at, v); });
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        int *last = reinterpret_cast<int *>(smem);
        if (t == 0)
            *last = (int)atomicAdd(a.count + s.adapter * gridDim.x + blockIdx.x, 1u) == k1 - k0 - 1;
        __syncthreads();
        if (!*last)
            return;
        for_results([&](int64_t at, f32x4 &v) {
            v = f32x4{0, 0, 0, 0};
            for (int k = k0; k < k1; k++)
                v += load_shared(a.part + k * size + at);
        });
    }
    for_results([&](int64_t at, f32x4 v) { *reinterpret_cast<f32x4 *>(out + at) = v; });
}

// Both gradients in one launch: the first `blocks` column blocks are A's (from
// the INT8 codes), the others B's (from dY, of type X).  QT >= 0: the rows of
// workgroups after the slabs' add dX's term to the product meanwhile (333 tokens,
// 4096 x 4096, rank 64 in fp32: 77 us for the call against 84 us with a launch of
// its own).
template <int X, int RB, int QT>
__global__ __launch_bounds__(256) void adapter_outer_kernel(OuterArgs a, OuterArgs b, int blocks, int slabs,
                                                            AdapterTermArgs e)
{
    constexpr int kX = terms_of(X) * TokenTile<outer_cols(X)>::kSize;
    constexpr int kCodes = TokenTile<outer_cols(X_I8)>::kSize;
    constexpr int kOuter = (kX > kCodes ? kX : kCodes) + 3 * TokenTile<RB * 16>::kSize;
    constexpr int kSize = QT >= 0 && 2 * kExpandTile > kOuter ? 2 * kExpandTile : kOuter;
    __shared__ __attribute__((aligned(16))) uint16_t smem[kSize];
    if constexpr (QT >= 0) {
        if ((int)blockIdx.y >= slabs) {
            const int64_t i = (int64_t)((int)blockIdx.y - slabs) * gridDim.x + blockIdx.x;
            const int64_t across = (e.C + 255) / 256;
            if (i < across * ((e.M + 15) / 16))
                expand<QT, true>(e, i % across, i / across, reinterpret_cast<float *>(smem));
            return;
        }
    }
    if ((int)blockIdx.x < blocks)
        outer_product<X_I8, false, RB>(a, blockIdx.x, smem);
    else
        outer_product<X, true, RB>(b, blockIdx.x - blocks, smem);
}

template <int X, int QT>
void run_outer(const OuterArgs &a, const OuterArgs &b, int slabs, const AdapterTermArgs &e, hipStream_t st)
{
    auto column_blocks = [](int64_t c, int cols) { return (c + cols - 1) / cols; };
    const int64_t blocks = column_blocks(a.C, outer_cols(X_I8)), wide = blocks + column_blocks(b.C, outer_cols(X));
    const int64_t terms = QT < 0 ? 0 : ((e.C + 255) / 256 * ((e.M + 15) / 16) + wide - 1) / wide;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)wide, (unsigned)(slabs + terms)), dim3(256), 0, st, a, b,
                           (int)blocks, slabs, e);
    };
    if (a.R <= 16)
        go(adapter_outer_kernel<X, 1, QT>);
    else if (a.R <= 32)
        go(adapter_outer_kernel<X, 2, QT>);
    else if (a.R <= 64)
        go(adapter_outer_kernel<X, 4, QT>);
    else
        go(adapter_outer_kernel<X, 8, QT>);
}

template <int X>
void run_outer(const OuterArgs &a, const OuterArgs &b, int slabs, const AdapterTermArgs *dx, hipStream_t st)
{
    if (!dx)
        run_outer<X, -1>(a, b, slabs, AdapterTermArgs{}, st);
    else if (dx->ad.bf16)
        run_outer<X, 1>(a, b, slabs, *dx, st);
    else
        run_outer<X, 4>(a, b, slabs, *dx, st);
}

// out[l] = the sum of l's slabs, in order; zeros for an adapter without tokens.
// Both gradients in one launch: the workgroups from the first sa / 1024 on are
// B's.
__global__ __launch_bounds__(256) void adapter_sum_kernel(const float *__restrict__ pa, int64_t sa,
                                                          float *__restrict__ da,
                                                          const float *__restrict__ pb, int64_t sb,
                                                          float *__restrict__ db,
                                                          const int32_t *__restrict__ first)
{
    const int64_t na = (sa + 1023) / 1024;
    const bool is_a = (int64_t)blockIdx.x < na;
    const float *part = is_a ? pa : pb;
    float *out = is_a ? da : db;
    const int64_t size = is_a ? sa : sb;
    const int64_t i = ((is_a ? blockIdx.x : blockIdx.x - na) * 256 + threadIdx.x) * 4;
    if (i >= size)
        return;
    const int64_t l = blockIdx.y;
    const int k0 = first[l], k1 = first[l + 1];
    f32x4 s = {0, 0, 0, 0};
#pragma unroll 4
    for (int k = k0; k < k1; k++)
        s += *reinterpret_cast<const f32x4 *>(part + k * size + i);
    *reinterpret_cast<f32x4 *>(out + l * size + i) = s;
}

} // namespace

static size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// A forward call's workspace: partial sums, terms.
size_t adapter_fwd_bytes(int64_t M, int64_t R)
{
    const size_t terms = (size_t)((M + 15) / 16) * terms_steps(0, (int)R) * 1024;
    return kPartBytes + terms;
}

const uint16_t *launch_adapter_u(const AdapterArgs &g, const int8_t *qx, const float *sx, float *u,
                                 unsigned *count, void *ws, hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    uint16_t *terms = reinterpret_cast<uint16_t *>(w + kPartBytes);
    const ShrinkArgs s{qx, sx, g.a, g.scale, g.ids, g.M, g.K, g.L, g.R, u, terms, g.bf16 ? 1 : 0, 1,
                       reinterpret_cast<float *>(w), count};
    g.bf16 ? run_shrink<X_I8, X_BF16>(s, st) : run_shrink<X_I8, X_F32>(s, st);
    return terms;
}

void launch_adapter_expand(const AdapterTermArgs &e, hipStream_t st)
{
    const dim3 grid((unsigned)((e.C + 255) / 256), (unsigned)((e.M + 15) / 16));
    if (e.ad.bf16)
        hipLaunchKernelGGL(adapter_expand_kernel<1>, grid, dim3(256), 0, st, e);
    else
        hipLaunchKernelGGL(adapter_expand_kernel<0>, grid, dim3(256), 0, st, e);
}

void launch_adapter_group(const int32_t *ids, int64_t M, int L, int32_t *order, int32_t *start,
                          hipStream_t st)
{
    hipLaunchKernelGGL(adapter_group_kernel, dim3(1), dim3(kGroupWaves * kWave), 0, st, ids, M, L, order,
                       start);
}

static int64_t slabs_of(int64_t M, int64_t L) { return M / kSlab + (M < L ? M : L); }

// So few tokens, hence slabs of one adapter, that the last to arrive adds them up.
// us for the call, 4096 x 4096, five adapters, added up in place / in a launch of
// their own, by tokens: rank 16 in bf16 333: 49/51, 700: 59/61, 1024: 65/66, 1500:
// 74/77, 2048: 93/90, 4096: 109/101; rank 64 in fp32 333: 59/64, 700: 74/78, 1024:
// 94/88, 1500: 112/111, 2048: 156/146.  No tokens at all: the launch writes the zeros.
static bool sums_in_place(int64_t M) { return M > 0 && M <= 4 * kSlab; }

// Column blocks of both gradients (a gradient's with the fewest columns each).
static int64_t outer_blocks(int64_t N, int64_t K)
{
    return (K + outer_cols(X_I8) - 1) / outer_cols(X_I8) + (N + outer_cols(X_F32) - 1) / outer_cols(X_F32);
}

// Offsets of a backward call's workspace.
struct BwdLayout {
    size_t part, bt, at, v, terms, table, first, count, pa, pb, end;
};

static BwdLayout bwd_layout(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    const size_t slabs = (size_t)slabs_of(M, L);
    const int pairs = terms_steps(3, (int)R), steps = pairs > terms_steps(4, (int)R) ? pairs : terms_steps(4, (int)R);
    BwdLayout o;
    o.part = 0;
    o.bt = round256(o.part + kPartBytes);
    o.at = round256(o.bt + (size_t)L * R * N * 6);
    o.v = round256(o.at + (size_t)L * (K / 16) * steps * 1024);
    o.terms = round256(o.v + (size_t)M * R * 4);
    o.table = round256(o.terms + (size_t)((M + 15) / 16) * steps * 1024);
    o.first = round256(o.table + slabs * sizeof(Slab));
    o.count = round256(o.first + ((size_t)L + 1) * 4);
    o.pa = round256(o.count + (sums_in_place(M) ? (size_t)L * outer_blocks(N, K) * 4 : 0));
    o.pb = round256(o.pa + slabs * (size_t)R * K * 4);
    o.end = round256(o.pb + slabs * (size_t)R * N * 4);
    return o;
}

size_t adapter_bwd_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    return bwd_layout(M, N, K, L, R).end;
}

AdapterEpilogue launch_adapter_bwd_v(const AdapterArgs &g, const void *dy, bool dy_bf16,
                                     const int32_t *start, float *da, float *db, unsigned *count,
                                     void *ws, hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    const BwdLayout o = bwd_layout(g.M, g.N, g.K, g.L, g.R);
    const PrepArgs p{g.a, g.b, reinterpret_cast<uint16_t *>(w + o.at), reinterpret_cast<uint16_t *>(w + o.bt),
                     g.N, g.K, g.M, g.L, g.R, adapter_term_apart(g.M, g.K) ? 4 : 3, (int)slabs_of(g.M, g.L), start,
                     reinterpret_cast<Slab *>(w + o.table), reinterpret_cast<int32_t *>(w + o.first),
                     sums_in_place(g.M) ? da : nullptr, sums_in_place(g.M) ? db : nullptr,
                     reinterpret_cast<unsigned *>(w + o.count),
                     sums_in_place(g.M) ? g.L * outer_blocks(g.N, g.K) : 0};
    const int64_t tiles = (int64_t)((g.R + 31) / 32) * ((g.N + 31) / 32 + (g.K + 31) / 32);
    const dim3 grid((unsigned)(g.M > 0 ? 1 + tiles : 1), (unsigned)g.L);
    if (g.bf16)
        hipLaunchKernelGGL(adapter_prep_kernel<true>, grid, dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(adapter_prep_kernel<false>, grid, dim3(256), 0, st, p);
    const ShrinkArgs s{dy,  nullptr, w + o.bt, g.scale, g.ids, g.M, g.N,
                       g.L, g.R,     reinterpret_cast<float *>(w + o.v),
                       reinterpret_cast<uint16_t *>(w + o.terms), g.bf16 ? 1 : p.qt, 1,
                       reinterpret_cast<float *>(w + o.part), count};
    if (g.M > 0) {
        if (dy_bf16)
            g.bf16 ? run_shrink<X_BF16, X_BF16>(s, st) : run_shrink<X_BF16, W_TERMS>(s, st);
        else
            g.bf16 ? run_shrink<X_F32, X_BF16>(s, st) : run_shrink<X_F32, W_TERMS>(s, st);
    }
    return AdapterEpilogue{s.out, s.terms, w + o.at, g.ids, g.L, g.R, g.bf16};
}

void launch_adapter_bwd_w(const AdapterArgs &g, const void *dy, bool dy_bf16, const int8_t *qx,
                          const float *sx, const float *u, const int32_t *order, float *da, float *db,
                          const AdapterTermArgs *dx, void *ws, hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    const BwdLayout o = bwd_layout(g.M, g.N, g.K, g.L, g.R);
    const int slabs = (int)slabs_of(g.M, g.L);
    const Slab *table = reinterpret_cast<const Slab *>(w + o.table);
    float *pa = reinterpret_cast<float *>(w + o.pa), *pb = reinterpret_cast<float *>(w + o.pb);
    const float *v = reinterpret_cast<const float *>(w + o.v);
    if (g.M > 0) {
        const bool here = sums_in_place(g.M);
        const int32_t *first = reinterpret_cast<const int32_t *>(w + o.first);
        unsigned *count = reinterpret_cast<unsigned *>(w + o.count);
        const OuterArgs a{v, sx, qx, order, table, g.M, g.K, g.R, pa, here ? da : nullptr, first, count};
        const OuterArgs b{u, nullptr, dy, order, table, g.M, g.N, g.R, pb, here ? db : nullptr, first, count};
        dy_bf16 ? run_outer<X_BF16>(a, b, slabs, dx, st) : run_outer<X_F32>(a, b, slabs, dx, st);
    }
    if (sums_in_place(g.M))
        return;
    const int64_t sa = (int64_t)g.R * g.K, sb = (int64_t)g.R * g.N;
    hipLaunchKernelGGL(adapter_sum_kernel, dim3((unsigned)((sa + 1023) / 1024 + (sb + 1023) / 1024), (unsigned)g.L),
                       dim3(256), 0, st, pa, sa, da, pb, sb, db,
                       reinterpret_cast<const int32_t *>(w + o.first));
}

} // namespace qlin
