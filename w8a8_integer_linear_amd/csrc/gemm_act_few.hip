// The forward products of a feed-forward block for tens of tokens, where the weight's
// bytes count and a 256 x 256 tile would be mostly empty (and for 16 tokens and fewer
// with a checkpoint, whose blocks are wider than the streaming kernel's rows).
#include "gemm_kernel.hpp"

namespace qlin {

namespace {

// act_value by a uniform switch: here the arithmetic after the sums is the smaller part.
__device__ __forceinline__ float act_of(int act, float z)
{
    switch (act) {
    case QLIN_ACT_RELU: return act_value<QLIN_ACT_RELU>(z);
    case QLIN_ACT_SILU: return act_value<QLIN_ACT_SILU>(z);
    case QLIN_ACT_GELU: return act_value<QLIN_ACT_GELU>(z);
    case QLIN_ACT_GELU_TANH: return act_value<QLIN_ACT_GELU_TANH>(z);
    default: return z;
    }
}

// A workgroup computes 16 TT tokens by 32 outputs (with a gate, 64 of the weight's rows:
// 32 of each half).  Its WAVES waves split the contraction: a chunk is WAVES steps of 64
// bytes of all those rows, copied by buffer-to-LDS loads of whole runs of a row
// (fragments loaded straight into registers, 64 bytes of 16 rows at a time, took up to
// twice as long: their rows lie at one offset of the memory channels), and wave w
// multiplies step w of each.  NB buffers: NB - 2 chunks are in flight while one is
// multiplied and the next lands.  Inside a row, 16-byte piece c sits at slot c ^ (row &
// 15).  The sums are added up in LDS (int32: any order gives the same) and finished
// eight outputs per lane.
template <int TT, bool GATED, int WAVES, int NB>
__global__ __launch_bounds__(WAVES * kWave) void few_act_kernel(GemmParams p)
{
    constexpr int H = GATED ? 2 : 1, WT = 2 * H;
    constexpr int kThreads = WAVES * kWave;
    constexpr int CHUNK = 64 * WAVES, kSlots = CHUNK / 16;
    constexpr int kAll = 16 * TT + 32 * H;          // rows of a chunk: x's, then the weight's
    constexpr int kBuf = kAll * CHUNK;
    constexpr int kLoads = kAll / 16;               // per wave and chunk, 1 KiB each
    constexpr int kRow = 32 * H + 1;        // words of a token's sums, odd: spread over the banks
    constexpr int kSums = 16 * TT * kRow * 4;
    static_assert(kSlots >= 16 && kSums <= NB * kBuf, "chunk shape");
    __shared__ __attribute__((aligned(1024))) int8_t smem[NB * kBuf];
    const int lane = __lane_id();
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int n0 = blockIdx.x * 32, m0 = blockIdx.y * 16 * TT;
    const int K = p.T, F = p.S, r = lane % 16, g = lane / 16;
    // Buffer resources that end where the arrays do: rows past the last are zeros.
    auto rows_from = [&](const int8_t *base, int64_t row, int64_t rows) {
        const int64_t left = (rows - row) * K;
        return make_rsrc(base + row * K, left < (int64_t)kOob ? (uint32_t)left : kOob);
    };
    const __amdgpu_buffer_rsrc_t xr = rows_from(p.a, m0, p.R);
    const __amdgpu_buffer_rsrc_t own = rows_from(p.b, n0, H * (int64_t)F);
    const __amdgpu_buffer_rsrc_t other = rows_from(p.b, n0 + (GATED ? F : 0), H * (int64_t)F);
    const int chunks = (K + CHUNK - 1) / CHUNK;
    auto issue = [&](int kc, int b) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int piece = (w * kLoads + i) * kWave;     // the instruction's first
            const int first = piece / kSlots;               // its first row
            const int row = (piece + lane) / kSlots, slot = (piece + lane) % kSlots;
            const int k = kc * CHUNK + (slot ^ (row & 15)) * 16;
            const int base = first < 16 * TT ? 0 : first < 16 * TT + 32 ? 16 * TT : 16 * TT + 32;
            const uint32_t off = k < K ? (uint32_t)((row - base) * K + k) : kOob;
            lds_i8 *dst = (lds_i8 *)smem + b * kBuf + piece * 16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                base == 0 ? xr : base == 16 * TT ? own : other,
                (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0, 0);
        }
    };
    i32x4 acc[TT][WT];
#pragma unroll
    for (int t = 0; t < TT; t++)
#pragma unroll
        for (int b = 0; b < WT; b++)
            acc[t][b] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < NB - 1; c++)
        issue(c, c);                                // (past the last chunk: zeros)
    int cur = 0, fill = NB - 1;
    for (int kc = 0; kc < chunks; kc++) {
        // Chunk kc has landed, and every wave has read chunk kc - 1 (its own LDS reads are
        // back), whose buffer is filled next.  (No fence, so that the loads stay in
        // flight.)
        wait_vmcnt<(NB - 2) * kLoads>();
        wait_lgkmcnt0();
        barrier_no_fence();
        issue(kc + NB - 1, fill);
        const int8_t *buf = smem + cur * kBuf;
        auto frag = [&](int row0) {
            const int row = row0 + r;
            return *reinterpret_cast<const i32x4 *>(buf + row * CHUNK + ((4 * w + g) ^ (row & 15)) * 16);
        };
        i32x4 v[WT], x[TT];
#pragma unroll
        for (int b = 0; b < WT; b++)
            v[b] = frag(16 * TT + 16 * b);
#pragma unroll
        for (int t = 0; t < TT; t++)
            x[t] = frag(16 * t);
        // The weight is the first operand: lane l has token l % 16 and, in register e,
        // row 4 (l / 16) + e.
#pragma unroll
        for (int t = 0; t < TT; t++)
#pragma unroll
            for (int b = 0; b < WT; b++)
                acc[t][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[b], x[t], acc[t][b], 0, 0, 0);
        cur = cur + 1 < NB ? cur + 1 : 0;
        fill = fill + 1 < NB ? fill + 1 : 0;
    }
    // (No load still writes to LDS, and no wave still reads the last chunk from it.)
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    barrier_no_fence();
    int32_t *sums = reinterpret_cast<int32_t *>(smem);
    for (int k = threadIdx.x; k < kSums / 4; k += kThreads)
        sums[k] = 0;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TT; t++)
#pragma unroll
        for (int b = 0; b < WT; b++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                atomicAdd(&sums[(16 * t + r) * kRow + 16 * b + 4 * g + e], acc[t][b][e]);
    __syncthreads();
    // Four lanes per token; the wave's lanes stay together (a checkpoint's block is four
    // neighbours'), those past the last row or column store nothing.
    const ActEpilogue &a = p.act;
    const int64_t N = H * (int64_t)F;
    const int per = (F + kCkBlock - 1) / kCkBlock;
    const int col = 8 * (threadIdx.x % 4);
    const bool col_ok = n0 + col < F;
    float cs[8 * H], bj[8 * H];
#pragma unroll
    for (int t = 0; t < 8 * H; t++) {
        const int64_t n = n0 + col + t % 8 + (t >= 8 ? (int64_t)F : 0);
        cs[t] = col_ok ? p.scol[n] : 0.0f;
        bj[t] = col_ok && p.bias ? p.bias[n] : 0.0f;
    }
    for (int row = threadIdx.x / 4; row < 16 * TT; row += kThreads / 4) {
        const int m = m0 + row;
        const bool ok = col_ok && m < p.R;
        const float rs = m < p.R ? p.srow[m] : 0.0f;
        float z[8 * H];
#pragma unroll
        for (int t = 0; t < 8 * H; t++) {
            // (Past the last column: 0, whatever the weight's next rows gave.)
            const int32_t sum = col_ok ? sums[row * kRow + col + t % 8 + (t >= 8 ? 32 : 0)] : 0;
            z[t] = (float)sum * rs * cs[t];
            if (p.bias)
                z[t] = z[t] + bj[t];
        }
        if (a.ck) {
#pragma unroll
            for (int h = 0; h < H; h++) {
                float s;
                const i32x2 c = ck_codes(z + 8 * h, s);
                if (ok) {
                    *reinterpret_cast<i32x2 *>(a.ck + m * N + h * (int64_t)F + n0 + col) = c;
                    if (col == 0)
                        a.ck_s[(int64_t)m * H * per + h * per + blockIdx.x] = s;
                }
            }
        }
        if (!ok)
            continue;
        const int64_t at = (int64_t)m * F + n0 + col;
        float y[8];
#pragma unroll
        for (int t = 0; t < 8; t++) {
            y[t] = act_of(a.act, z[t]);
            if constexpr (GATED)
                y[t] = y[t] * z[8 + t];
        }
        if (!GATED && a.res) {
            float q[8];
            if (a.res_bf16)
                load8<true>(a.res, at, q);
            else
                load8<false>(a.res, at, q);
#pragma unroll
            for (int t = 0; t < 8; t++)
                y[t] = y[t] + q[t];
        }
        if (a.y_bf16)
            *reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(p.out) + at) = pack_bf16x8(y);
        else
            store8(static_cast<float *>(p.out), at, y);
    }
}

} // namespace

// Whether the tiles above serve a call better than 256 x 256 ones: up to 64 tokens,
// and up to 512 tiles of 128 tokens by 32 of the weight's rows.  us, these / those:
//   14336 x 4096 gated   64 tokens 37 / 47, 100 tokens (896 tiles) 52 / 47
//   7168 x 4096          128 (224) 17 / 36, 256 (448) 30 / 38, 512 (896) 60 / 44
//   4096 x 14336         128 (128) 27 / 74, 256 (256) 43 / 82
//   2048 x 5376          256 (128) 10.5 / 36
bool product_act_few(const ProductArgs &a)
{
    return a.M <= 64 || (a.N + 31) / 32 * ((a.M + 127) / 128) <= 512;
}

void launch_product_act_few(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    GemmParams p = gemm_params(a);
    p.act = e;
    p.S = (int)e.F;
    auto tiles = [&](int tokens) { return (e.F + 31) / 32 * ((a.M + tokens - 1) / tokens); };
    auto go = [&](auto kernel, int tokens, int waves) {
        const dim3 grid((unsigned)((e.F + 31) / 32), (unsigned)((a.M + tokens - 1) / tokens));
        hipLaunchKernelGGL(kernel, grid, dim3(waves * kWave), 0, st, p);
    };
    // The most tokens per workgroup that leave nearly one per compute unit: fewer make
    // more of them, which each read the same weight (7168 x 4096, 64 tokens, 64 or 32 per
    // workgroup: 12.1 / 16.0 us; 4096 x 14336: 28.3 / 20.5).  Eight waves and longer
    // runs where one workgroup is all that a compute unit has (4096 x 14336, 128 tokens:
    // 28.6 -> 26.7 us).
    constexpr int kEnough = 200;
    auto with = [&](auto gated) {
        constexpr bool G = decltype(gated)::value;
        if (a.M > 64 && tiles(128) >= kEnough) {
            go(few_act_kernel<8, G, 4, 3>, 128, 4);
        } else if (a.M > 32 && tiles(64) >= kEnough) {
            if constexpr (G)
                go(few_act_kernel<4, G, 4, 3>, 64, 4);
            else if (tiles(64) > kRound)
                go(few_act_kernel<4, G, 4, 3>, 64, 4);
            else
                go(few_act_kernel<4, G, 8, 3>, 64, 8);
        } else if (a.M > 16) {
            go(few_act_kernel<2, G, 8, 3>, 32, 8);
        } else {
            go(few_act_kernel<1, G, 8, 3>, 16, 8);
        }
    };
    if (e.gated)
        with(std::true_type());
    else
        with(std::false_type());
}

} // namespace qlin
