// The forward products of a feed-forward block: bias, activation and residual, or
// the gate, and the 8-bit checkpoint of the sums in the epilogue.  One instance per
// activation (a switch in the epilogue would hold all of them in the instruction
// cache); types, residual and checkpoint are uniform branches there.
#include "gemm_kernel.hpp"

namespace qlin {

namespace {

template <int EPI> void run_tiles(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    GemmParams p = gemm_params(a);
    p.act = e;
    p.S = (int)e.F;
    p.tiles_i = (p.R + 255) / 256;
    p.tiles_j = (int)((a.N + 255) / 256);       // (with a gate, 128 outputs per tile)
    const int tiles = p.tiles_i * p.tiles_j;
    const dim3 block(8 * kWave);
    if (p.split >= 2 && act_split_plan(a.M, a.N, a.K).split >= 2)
        hipLaunchKernelGGL((gemm_kernel<2, 4, false, false, EPI, MODE_SPLIT>),
                           dim3((unsigned)(p.full + (tiles - p.full) * p.split)), block, 0, st, p);
    else
        hipLaunchKernelGGL((gemm_kernel<2, 4, false, false, EPI, MODE_PLAIN>), dim3((unsigned)tiles),
                           block, 0, st, p);
}

// The product for M <= 16 tokens: the weight is streamed once, which bounds it (a bare
// read of 117 MB from memory takes 18.8 us, of 59 MB 10.2; this 23.0 for 3 tokens, 13.9
// for 5; with the weight in the infinity cache 15.9, 9.0; 18.6, 11.6).  A workgroup
// owns ROWS of its rows, with a gate ROWS / 2 of each half, and copies them CHUNK bytes
// of each at a time into LDS by buffer-to-LDS loads, two chunks in flight, and with
// them the tokens' values of the chunk into registers.  Inside a row, 16-byte piece c
// sits at slot c ^ (row & 15), so that the MFMA reads of 16 rows at one offset fall on
// distinct banks.  The four waves split a chunk's steps of 64 bytes, one
// v_mfma_i32_16x16x64_i8 each per 16 rows with the (zero-padded) 16 tokens, and combine
// their sums through LDS; then thread t has token t / 16 and every 16th output.
template <int CHUNK, int ROWS, int EPI>
__global__ __launch_bounds__(256) void stream_act_kernel(GemmParams p)
{
    constexpr bool kGated = EPI >= EPI_GATED;
    constexpr int kOut = kGated ? ROWS / 2 : ROWS;  // outputs of a workgroup
    constexpr int kBuf = ROWS * CHUNK;              // one chunk of the rows
    constexpr int kSlots = CHUNK / 16;              // 16-byte pieces of a row's chunk
    constexpr int kLoads = kBuf / 4096;             // per wave and chunk, 1 KiB each
    constexpr int kSteps = CHUNK / 256;             // MFMA steps per wave and chunk
    constexpr int kTiles = ROWS > 16 ? ROWS / 16 : 1;
    static_assert(kBuf % 4096 == 0 && CHUNK % 256 == 0, "chunk shape");
    // (One LDS object, so that reads of one buffer do not wait for the loads that fill
    // the other.)
    constexpr int kRed = kTiles * 4 * kWave * 16;
    __shared__ __attribute__((aligned(1024))) int8_t smem[2 * kBuf > kRed ? 2 * kBuf : kRed];
    const int lane = __lane_id();
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int n0 = blockIdx.x * kOut, M = p.R, K = p.T;
    const int col = lane % 16, g = lane / 16;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.a);
    const int8_t *own = p.b + (int64_t)n0 * K, *other = own + p.act.F * K;
    const int chunks = (K + CHUNK - 1) / CHUNK;

    // Chunk kc into buffer b, and this wave's x of it, from L2 (bytes past K and rows
    // past M are zeros).
    auto issue = [&](int kc, int b, i32x4 (&av)[kSteps]) {
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int piece = (w * kLoads + i) * kWave;     // the instruction's first
            const int row = (piece + lane) / kSlots, slot = (piece + lane) % kSlots;
            const bool up = kGated && piece / kSlots >= kOut;
            const int k = kc * CHUNK + (slot ^ (row & 15)) * 16;
            const uint32_t off = kc < chunks && k < K ? (uint32_t)((row - (up ? kOut : 0)) * K + k) : kOob;
            lds_i8 *dst = (lds_i8 *)smem + b * kBuf + piece * 16;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                make_rsrc(up ? other : own), (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0,
                0);
        }
#pragma unroll
        for (int t = 0; t < kSteps; t++) {
            const int k = kc * CHUNK + (w + 4 * t) * 64 + g * 16;
            av[t] = __builtin_amdgcn_raw_buffer_load_b128(
                xr, kc < chunks && k < K && col < M ? (uint32_t)(col * K + k) : kOob, 0, 0);
        }
    };
    i32x4 acc[kTiles];
#pragma unroll
    for (int q = 0; q < kTiles; q++)
        acc[q] = i32x4{0, 0, 0, 0};
    auto multiply = [&](int b, const i32x4 (&av)[kSteps]) {
        const int8_t *buf = smem + b * kBuf;
#pragma unroll
        for (int t = 0; t < kSteps; t++)
#pragma unroll
            for (int q = 0; q < kTiles; q++) {
                const int piece = (w + 4 * t) * 4 + g, row = 16 * q + col % (ROWS < 16 ? ROWS : 16);
                const i32x4 bv =
                    *reinterpret_cast<const i32x4 *>(buf + row * CHUNK + (piece ^ (row & 15)) * 16);
                acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[t], bv, acc[q], 0, 0, 0);
            }
    };
    // Per chunk: the next one's loads (of nothing past the last), a wait until only they
    // are outstanding, the products; the second barrier, behind a wait for the wave's
    // own LDS reads, holds the buffer until every wave has read it.  (No fences, so that
    // the loads stay in flight.)
    i32x4 x0[kSteps], x1[kSteps];
    issue(0, 0, x0);
    for (int kc = 0; kc < chunks; kc += 2) {
        issue(kc + 1, 1, x1);
        wait_vmcnt<kLoads + kSteps>();
        barrier_no_fence();
        multiply(0, x0);
        wait_lgkmcnt0();
        barrier_no_fence();
        issue(kc + 2, 0, x0);
        wait_vmcnt<kLoads + kSteps>();
        barrier_no_fence();
        multiply(1, x1);
        wait_lgkmcnt0();
        barrier_no_fence();
    }
    // (The loads of nothing past the end still write zeros to LDS.)
    wait_vmcnt<0>();
    barrier_no_fence();
    // Lane l, register r of a sum: token 4 (l / 16) + r, row l % 16.
    i32x4 *red = reinterpret_cast<i32x4 *>(smem);
#pragma unroll
    for (int q = 0; q < kTiles; q++)
        red[(q * 4 + w) * kWave + lane] = acc[q];
    __syncthreads();
    const int m = threadIdx.x / 16;
    if (m >= M)
        return;
    auto z = [&](int row, int64_t n) {
        int32_t sum = 0;
#pragma unroll
        for (int i = 0; i < 4; i++)
            sum += reinterpret_cast<const int32_t *>(
                red)[((row / 16 * 4 + i) * kWave + 16 * (m / 4) + row % 16) * 4 + m % 4];
        const float f = (float)sum * p.srow[m] * p.scol[n];
        return p.bias ? f + p.bias[n] : f;
    };
    const ActEpilogue &e = p.act;
#pragma unroll
    for (int c = threadIdx.x % 16; c < kOut; c += 16) {
        const int64_t at = (int64_t)m * e.F + n0 + c;
        float y = act_value<EPI % EPI_ACT>(z(c, n0 + c));
        if constexpr (kGated)
            y = y * z(kOut + c, n0 + c + e.F);
        if (e.res)
            y = y + (e.res_bf16 ? bf16_lo(static_cast<const uint16_t *>(e.res)[at])
                                : static_cast<const float *>(e.res)[at]);
        if (e.y_bf16)
            static_cast<uint16_t *>(p.out)[at] = (uint16_t)pack_bf16x2(y, y);
        else
            static_cast<float *>(p.out)[at] = y;
    }
}

template <int EPI> void run_stream(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    GemmParams p = gemm_params(a);
    p.act = e;
    auto go = [&](auto kernel, int rows) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.N / rows)), dim3(256), 0, st, p);
    };
    // 16 rows in chunks of 1 KiB, four workgroups per compute unit.  Every workgroup
    // reads all of x from L2, which from 8 tokens on takes as long as the weight: 32
    // rows then, where that leaves enough workgroups (us for 16 tokens with 16 / 32
    // rows: 28672 x 4096 30.5 / 26.5, 14336 x 4096 18.5 / 14.4, 7168 x 5376 12.4 / 11.6,
    // 4096 x 4096 8.0 / 8.7; 5 tokens, 28672 x 4096: 23.7 / 26.0).  Few tokens and few
    // workgroups: 8 rows (4096 x 4096, two tokens: 7.2 -> 6.2; eight tokens, contraction
    // 14336: 13.7 -> 15.0).
    if (a.M > 8 && a.N % 32 == 0 && a.N >= 32 * 200)
        go(stream_act_kernel<512, 32, EPI>, 32);
    else if (a.M <= 4 && a.N / 16 <= kRound)
        go(stream_act_kernel<1024, 8, EPI>, 8);
    else
        go(stream_act_kernel<1024, 16, EPI>, 16);
}

template <int ACT> void run(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    // (A workgroup of the streaming kernel may have 16 of the weight's rows, less than a
    // block of the checkpoint.)
    const bool stream = a.M <= 16 && !e.ck;
    if (!stream && product_act_few(a))
        return launch_product_act_few(a, e, st);
    if (e.gated)
        stream ? run_stream<EPI_GATED + ACT>(a, e, st) : run_tiles<EPI_GATED + ACT>(a, e, st);
    else
        stream ? run_stream<EPI_ACT + ACT>(a, e, st) : run_tiles<EPI_ACT + ACT>(a, e, st);
}

} // namespace

// The last round's tiles are split along the contraction where that saves more than
// their partial sums cost, which grows with the tiles (all of them write theirs at
// once).  us split / whole, bf16 with GELU, by tiles and contraction:
//               2048          4096          8192
//     32     59.6 / 61.2  85.4 / 97.2
//     64     31.3 / 30.0  39.6 / 45.3   57.4 / 75.8
//    112     38.1 / 31.0  46.7 / 45.8   65.6 / 75.9
//    128     41.4 / 32.7  51.0 / 48.3   71.5 / 77.1
SplitPlan act_split_plan(int64_t M, int64_t N, int64_t K)
{
    const SplitPlan none{0, 0, 1};
    ProductArgs a{};
    a.M = M;
    a.N = N;
    if (M <= 16 || product_act_few(a))
        return none;
    const SplitPlan sp = split_plan(0, M, N, K);
    return 10 * ((K + 127) / 128) > 3 * (int64_t)sp.tail ? sp : none;
}

void launch_product_act(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    switch (e.act) {
    case QLIN_ACT_NONE: return run<QLIN_ACT_NONE>(a, e, st);
    case QLIN_ACT_RELU: return run<QLIN_ACT_RELU>(a, e, st);
    case QLIN_ACT_SILU: return run<QLIN_ACT_SILU>(a, e, st);
    case QLIN_ACT_GELU: return run<QLIN_ACT_GELU>(a, e, st);
    default: return run<QLIN_ACT_GELU_TANH>(a, e, st);
    }
}

} // namespace qlin
