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
    if (p.split >= 2)
        hipLaunchKernelGGL((gemm_kernel<2, 4, false, false, EPI, MODE_SPLIT>),
                           dim3((unsigned)(p.full + (tiles - p.full) * p.split)), block, 0, st, p);
    else
        hipLaunchKernelGGL((gemm_kernel<2, 4, false, false, EPI, MODE_PLAIN>), dim3((unsigned)tiles),
                           block, 0, st, p);
}

template <int EPI> void run_stream(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.N / 16)), dim3(256), 0, st, a.a, a.srow, a.b, a.scol,
                           a.bias, (int)a.M, (int)e.F, (int)a.K, a.out, e);
    };
    if (a.N / 16 > kRound)
        go(skinny_fwd_kernel<false, 1024, -1, EPI>);
    else
        go(skinny_fwd_kernel<false, 4096, -1, EPI>);
}

template <int ACT> void run(const ProductArgs &a, const ActEpilogue &e, hipStream_t st)
{
    // (A workgroup of the streaming kernel has 16 of the weight's rows, less than a
    // block of the checkpoint.)
    const bool stream = a.M <= 16 && !e.ck;
    if (e.gated)
        stream ? run_stream<EPI_GATED + ACT>(a, e, st) : run_tiles<EPI_GATED + ACT>(a, e, st);
    else
        stream ? run_stream<EPI_ACT + ACT>(a, e, st) : run_tiles<EPI_ACT + ACT>(a, e, st);
}

} // namespace

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
