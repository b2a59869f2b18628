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
// units.  One bound for both directions and every rank; us for the call with the
// term apart / in the epilogues, contraction 4096, by tiles (611 and 2048 tokens):
//                              48      84        120       128       144       192
//   forward, rank 16, bf16   50/52   57/55   63/58 (108)  74/62     67/59     72/60
//   forward, rank 64, fp32   66/73   77/76   85/80 (108) 110/88     95/82    105/84
//   dX, rank 16, bf16                66/72     79/80      91/89     81/80     88/82
//   dX, rank 64, bf16                91/101   109/109    133/121   116/111   133/114
//   dX, rank 64, fp32                87/125   100/133    126/146   106/136   119/140
// (32 tiles, 333 tokens, dX: 49/65, 63/97, 60/126.)  So the forward changes sides at
// about 84 tiles, dX at about 130, but dX with fp32 adapters of rank 64, whose six
// pairs of terms the epilogues read, only at about 256 (192/183): between the bound
// and there it takes up to half as long again as with the term apart.
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
