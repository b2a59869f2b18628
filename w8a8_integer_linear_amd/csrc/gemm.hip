// The products of the layer: their kernels' instances and launches (the
// kernels themselves are in gemm_kernel.hpp).
#include "gemm_kernel.hpp"

namespace qlin {

namespace {

// Zero fill of n 32-bit words (arrival counters), a kernel rather than a
// memset so that it can sit in a captured graph.
__global__ __launch_bounds__(256) void zero_words_kernel(uint32_t *p, int n)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n)
        p[i] = 0;
}

template <int WM, int WN, bool AKM, bool BKM, int EPI>
void run_gemm(const GemmParams &p0, hipStream_t st)
{
    GemmParams p = p0;
    p.tiles_i = (p.R + 255) / 256;
    p.tiles_j = (p.S + 255) / 256;
    const int tiles = p.tiles_i * p.tiles_j;
    const dim3 block(WM * WN * kWave);
    if (p.ws_mode != 0) {
        if constexpr (EPI != EPI_RAW)
            hipLaunchKernelGGL((gemm_kernel<WM, WN, AKM, BKM, EPI, MODE_CHUNK>), dim3(tiles), block,
                               0, st, p);
    } else if (p.split >= 2) {
        const unsigned grid = (unsigned)(p.full + (tiles - p.full) * p.split);
        if constexpr (EPI != EPI_RAW)
            hipLaunchKernelGGL((gemm_kernel<WM, WN, AKM, BKM, EPI, MODE_SPLIT>), dim3(grid), block,
                               0, st, p);
    } else {
        hipLaunchKernelGGL((gemm_kernel<WM, WN, AKM, BKM, EPI, MODE_PLAIN>), dim3(tiles), block, 0,
                           st, p);
    }
}

// Tile configuration of the three products: 256 x 256 outputs per
// workgroup, 8 waves each owning 128 x 64, 128 contraction bytes per stage
// (two stages in flight in 128 KiB of LDS).
template <bool AKM, bool BKM, int EPI>
void run_cfg(const GemmParams &p, hipStream_t st)
{
    run_gemm<2, 4, AKM, BKM, EPI>(p, st);
}

} // namespace

SplitPlan split_plan(int op, int64_t M, int64_t N, int64_t K)
{
    SplitPlan none{0, 0, 1};
    if (op == 0 && M <= 16)
        return none;    // weight-streaming kernel
    const int64_t R = op == 2 ? N : M, S = op == 0 ? N : K, T = op == 0 ? K : (op == 1 ? N : M);
    const int64_t tiles = ((R + 255) / 256) * ((S + 255) / 256);
    const int64_t full = tiles / kRound * kRound, tail = tiles - full;
    if (tail == 0)
        return none;
    int64_t split = kRound / tail;
    const int64_t by_len = ((T + 127) / 128) / kMinPieceStages;
    split = split < by_len ? split : by_len;
    split = split < kMaxPieces ? split : kMaxPieces;
    if (split == 3 && tail * split > kMaxThreeWayUnits)
        split = 2;
    if (split < 2)
        return none;
    return SplitPlan{(int)full, (int)tail, (int)split};
}

// Contraction terms per launch of a chunked product (1023 stages of 128):
// within the int32-exact bound of 131,071.
constexpr int64_t kChunkLen = 1023 * 128;

bool product_addressable(int op, int64_t M, int64_t N, int64_t K)
{
    const int64_t T = op == 0 ? K : (op == 1 ? N : M);
    const int64_t t = T > 131071 ? kChunkLen : T;       // contraction of one launch
    auto lo = [](int64_t a, int64_t b) { return a < b ? a : b; };
    // Row operand of 'rows' rows with stride ld: a tile's loads reach
    // (rows in the tile - 1) * ld + t bytes past its base.  Km operand with
    // stride ld: a stage's loads reach (contraction rows in the stage - 1) *
    // ld + 256 (one tile's columns).
    auto row_ok = [&](int64_t rows, int64_t ld) {
        return rows < 1 || (lo(rows, 256) - 1) * ld + t <= (int64_t)kOob;
    };
    auto km_ok = [&](int64_t ld) { return t < 1 || (lo(t, 128) - 1) * ld + 256 <= (int64_t)kOob; };
    if (op == 0)
        return row_ok(M, K) && row_ok(N, K);
    if (op == 1)
        return row_ok(M, N) && km_ok(K);
    return km_ok(N) && km_ok(K);
}

void launch_zero_words(void *p, int n, hipStream_t st)
{
    if (n > 0)
        hipLaunchKernelGGL(zero_words_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st,
                           static_cast<uint32_t *>(p), n);
}

size_t split_ws_bytes(const SplitPlan &sp)
{
    if (sp.split < 2)
        return 0;
    return kSplitCountBytes + (size_t)sp.tail * sp.split * 256 * 256 * sizeof(int32_t);
}

void launch_product(const ProductArgs &a, hipStream_t st)
{
    GemmParams p = gemm_params(a);
    if (a.op == 0) {
        if (a.M <= 16 && a.ws_mode == 0) {
            auto go = [&](auto kernel) { run_skinny(kernel, a, AdapterEpilogue{}, st); };
            const bool wide = a.N / 16 > kRound;
            if (a.raw)
                wide ? go(skinny_fwd_kernel<true, 1024>) : go(skinny_fwd_kernel<true, 4096>);
            else
                wide ? go(skinny_fwd_kernel<false, 1024>) : go(skinny_fwd_kernel<false, 4096>);
            return;
        }
        if (a.raw)
            run_cfg<false, false, EPI_RAW>(p, st);
        else
            run_cfg<false, false, EPI_FWD>(p, st);
    } else if (a.op == 1) {
        if (a.raw) {
            run_cfg<false, true, EPI_RAW>(p, st);
        } else if (a.had >= 2 && a.had <= 128) {
            // dX with the un-rotation in the epilogue.
            p.had = a.had;
            p.had_scale = a.had_scale;
            run_cfg<false, true, EPI_ROWSCALE_HAD>(p, st);
        } else {
            run_cfg<false, true, EPI_ROWSCALE>(p, st);
        }
    } else {
        if (a.raw)
            run_cfg<true, true, EPI_RAW>(p, st);
        else
            run_cfg<true, true, EPI_ROWSCALE>(p, st);
    }
}

// Products whose contraction exceeds the int32-exact bound: chunks of 1023
// stages (130,944 terms, within the bound) run as ordinary products on the
// operands' sub-ranges; the first stores its int32 sums into the int64
// workspace, the middle ones add theirs, and the last one's epilogue takes
// acc + workspace through the usual dequant (and rotation) arithmetic.
void launch_product_long(const ProductArgs &a, int64_t *ws, hipStream_t st)
{
    const int64_t T = a.op == 0 ? a.K : (a.op == 1 ? a.N : a.M);
    for (int64_t k0 = 0; k0 < T; k0 += kChunkLen) {
        ProductArgs c = a;
        const int64_t len = T - k0 < kChunkLen ? T - k0 : kChunkLen;
        c.t_len = len;
        c.ws = ws;
        c.ws_mode = k0 == 0 ? 1 : (k0 + len >= T ? 3 : 2);
        if (a.op == 0) {
            c.a = a.a + k0;
            c.b = a.b + k0;
        } else if (a.op == 1) {
            c.a = a.a + k0;
            c.b = a.b + k0 * a.K;
        } else {
            c.a = a.a + k0 * a.N;
            c.b = a.b + k0 * a.K;
        }
        launch_product(c, st);
    }
}

} // namespace qlin
