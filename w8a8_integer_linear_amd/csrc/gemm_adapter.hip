// The forward and dX products with a low-rank term in their epilogues: each
// token's adapter is added to the outputs before they are first written, so
// the adapters cost no pass over y or dx (reading and writing y once more took
// 72 us of 546 at 12000 x 5376 -> 7168).
#include "gemm_kernel.hpp"

namespace qlin {

namespace {

template <bool BKM, int EPI> void run(GemmParams &p, hipStream_t st)
{
    p.tiles_i = (p.R + 255) / 256;
    p.tiles_j = (p.S + 255) / 256;
    const int tiles = p.tiles_i * p.tiles_j;
    const dim3 block(8 * kWave);
    if (p.split >= 2)
        hipLaunchKernelGGL((gemm_kernel<2, 4, false, BKM, EPI, MODE_SPLIT>),
                           dim3((unsigned)(p.full + (tiles - p.full) * p.split)), block, 0, st, p);
    else
        hipLaunchKernelGGL((gemm_kernel<2, 4, false, BKM, EPI, MODE_PLAIN>), dim3((unsigned)tiles),
                           block, 0, st, p);
}

} // namespace

// Few tiles: added in the epilogues, the term would be the work of as few compute
// units (backward of 333 tokens, 4096 x 4096, rank 64 in fp32: 141 us against 77
// us with the term apart; forward of 611 tokens, 4096 -> 14336, rank 32, 168
// tiles: 73 us against 98 us).
bool adapter_term_apart(int64_t rows, int64_t cols)
{
    return ((rows + 255) / 256) * ((cols + 255) / 256) < 128;
}

void launch_product_adapter(const ProductArgs &a, const AdapterEpilogue &ad, hipStream_t st)
{
    if (a.op == 0 && a.M <= 16) {
        auto go = [&](auto kernel) { run_skinny(kernel, a, ad, st); };
        const bool wide = a.N / 16 > kRound;
        if (ad.bf16)
            wide ? go(skinny_fwd_kernel<false, 1024, X_BF16>) : go(skinny_fwd_kernel<false, 4096, X_BF16>);
        else
            wide ? go(skinny_fwd_kernel<false, 1024, X_F32>) : go(skinny_fwd_kernel<false, 4096, X_F32>);
        return;
    }
    GemmParams p = gemm_params(a);
    p.ad = ad;
    if (a.op == 0) {
        if (adapter_term_apart(p.R, p.S)) {
            launch_product(a, st);
            launch_adapter_expand({ad, p.R, p.S, static_cast<float *>(a.out), 0, 1.0f}, st);
            return;
        }
        ad.bf16 ? run<false, EPI_FWD_ADAPTER_BF16>(p, st) : run<false, EPI_FWD_ADAPTER_F32>(p, st);
    } else {
        // (A block of 1: no rotation, or one that follows in a launch of its own.)
        p.had = a.had >= 2 && a.had <= 128 ? a.had : 1;
        p.had_scale = p.had > 1 ? a.had_scale : 1.0f;
        ad.bf16 ? run<true, EPI_HAD_ADAPTER_BF16>(p, st) : run<true, EPI_HAD_ADAPTER_TERMS>(p, st);
    }
}

} // namespace qlin
