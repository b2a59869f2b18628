// Host-side launchers of the qlin kernels.  Arguments are validated by the
// C-ABI layer (api.hip) before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlin {

void launch_quantize_rows(const void *x, bool bf16, int64_t rows, int64_t cols,
                          const float *prescale, int had, float cb, int8_t *q, float *s,
                          hipStream_t st);

void launch_quantize_cols(const void *x, bool bf16, int64_t rows, int64_t cols,
                          const float *prescale, int8_t *q, float *s, float *col_sum,
                          hipStream_t st);

// Both quantizations of the output gradient: rows of x * sw -> (q1, s1),
// columns of x * sx -> (q2, s2) and the column sums of x.  q2 serves as
// scratch for the row and column partials before its codes are written.
void launch_quantize_grad(const void *x, bool bf16, int64_t rows, int64_t cols, const float *sw,
                          const float *sx, int8_t *q1, float *s1, int8_t *q2, float *s2,
                          float *col_sum, hipStream_t st);

void launch_dequantize_weight(const int8_t *q, const float *sw, int64_t rows, int64_t cols,
                              int blk, float cb, float *w, hipStream_t st);

void launch_hadamard(const void *x, bool bf16, int64_t rows, int64_t cols, int blk, float cb,
                     float *y, hipStream_t st);

// Products.  op: 0 forward, 1 dX, 2 dW.  epi: 0 raw int32, 1 dequant.
struct ProductArgs {
    int op;
    const int8_t *a;
    const int8_t *b;
    int64_t M, N, K;
    const float *srow;  // sx, sg1 or sg2
    const float *scol;  // sw (forward only)
    const float *bias;  // forward only, may be null
    void *out;          // float* or int32_t*
    bool raw;           // int32 accumulators instead of dequantized floats
    int had = 0;        // dX only: rotate each output row in blocks of 'had' (<= 128)
    float had_scale = 1.0f;
    int64_t t_len = 0;        // contraction length of this launch (0: the full one)
    int64_t *ws = nullptr;    // int64 running sums of a split contraction
    int ws_mode = 0;          // 0 none, 1 store, 2 add, 3 finish from acc + ws
    // Workspace for balancing the last round of tiles (split_plan): arrival
    // counters in its first kSplitCountBytes (zero on entry, zero on exit),
    // then the pieces' int32 partial sums.  Null: no balancing.
    void *split_ws = nullptr;
};

void launch_product(const ProductArgs &p, hipStream_t st);

// The low-rank term of a product's output row i: sum_r p[i, r] q[ids[i], j, r]
// with p [rows, R] fp32 and q [L, cols, R] bf16 or, in the forward product, fp32;
// the dX product takes an fp32 q as bf16 terms, as adapter_prep_kernel makes
// them.  terms holds p as such terms, in the layout of adapter_frag.hpp that goes
// with q's form (the forward product of 16 rows or fewer reads p instead).
struct AdapterEpilogue {
    const float *p;
    const uint16_t *terms;
    const void *q;
    const int32_t *ids;
    int L, R;
    bool bf16;
};
// A forward or dX product (no workspace mode, contraction within the int32
// bound) with that term added; a dX product only where adapter_term_apart is
// false.
void launch_product_adapter(const ProductArgs &p, const AdapterEpilogue &ad, hipStream_t st);
// Whether that term has a launch of its own, for outputs of this size.
bool adapter_term_apart(int64_t rows, int64_t cols);
// The term added to outputs [M, C] in memory: a forward product's in a launch of
// its own; dX's, whose sums are then rotated in blocks of had (2 .. 128; 0: not),
// with the adapters' gradients (launch_adapter_bwd_w).
struct AdapterTermArgs {
    AdapterEpilogue ad;
    int64_t M, C;
    float *out;
    int had;
    float cb;
};
void launch_adapter_expand(const AdapterTermArgs &e, hipStream_t st);

// What a forward product's outputs z become in the kernel: y = act(z) + residual
// [M, F], or with a gate act(z[:, :F]) z[:, F:]; and the checkpoint of z, INT8
// codes [M, N] with a scale per kCkBlock outputs of a row (of each half, the last
// one's block may be short).  N = F, or 2 F with a gate (ProductArgs::N).
constexpr int kCkBlock = 32;
struct ActEpilogue {
    int act;
    bool gated;
    int64_t F;
    bool y_bf16;
    const void *res;        // may be null
    bool res_bf16;
    int8_t *ck;             // may be null
    float *ck_s;
};
// ProductArgs::out is y.
void launch_product_act(const ProductArgs &p, const ActEpilogue &e, hipStream_t st);
// The same in tiles of few tokens, and whether they serve a call better
// (gemm_act_few.hip).
bool product_act_few(const ProductArgs &p);
void launch_product_act_few(const ProductArgs &p, const ActEpilogue &e, hipStream_t st);

// Backward of act and gate from the checkpoint (act_bwd.hip).
struct ActBackward {
    const void *dy;
    bool dy_bf16;
    const int8_t *ck;
    const float *ck_s;
    int act;
    bool gated;
    const float *sw, *sx;   // of the two quantizations; null with s1, s2
    int64_t M, F;
    void *dz;
    bool dz_bf16;
    float *s1, *s2, *db;    // may be null
};
size_t act_bwd_bytes(int64_t M, int64_t F, bool gated);
void launch_act_bwd(const ActBackward &a, void *ws, hipStream_t st);

// The codes of both quantizations of a gradient whose scales are known.
void launch_grad_codes(const void *x, bool bf16, int64_t rows, int64_t cols, const float *sw,
                       const float *sx, const float *s1, const float *s2, int8_t *q1, int8_t *q2,
                       hipStream_t st);

// Whether the product kernels can address every operand byte of this shape
// with their 32-bit buffer offsets (for contractions past the int32 bound,
// those of one chunk's launch).
bool product_addressable(int op, int64_t M, int64_t N, int64_t K);

// How a product balances its last round of 256 x 256 tiles over the chip:
// 'full' whole tiles, then each of the 'tail' remaining tiles in 'split'
// pieces along the contraction (split 1: no balancing).
struct SplitPlan {
    int full, tail, split;
};
constexpr size_t kSplitCountBytes = 4096;
SplitPlan split_plan(int op, int64_t M, int64_t N, int64_t K);
// Of launch_product_act's calls (gemm_act.hip).
SplitPlan act_split_plan(int64_t M, int64_t N, int64_t K);
// Workspace bytes the plan needs (0 when it splits nothing).
size_t split_ws_bytes(const SplitPlan &sp);
// Zero n 32-bit words at p on the stream (a kernel, so graph capture holds
// no memset node).
void launch_zero_words(void *p, int n, hipStream_t st);

// A product whose contraction exceeds the int32 bound, in chunks combined in
// the int64 workspace ws [rows, cols] (8 bytes per output).
void launch_product_long(const ProductArgs &p, int64_t *ws, hipStream_t st);

// Streaming device copy of nbytes (a multiple of 16) between 16-byte aligned
// buffers: the reference for the memory-bound kernels' bandwidth.
void launch_stream_copy(const void *src, void *dst, int64_t nbytes, hipStream_t st);

// Matrix-core ceiling: `workgroups` workgroups of 8 waves repeat the
// products' MFMA sequence `iters` times on kMfmaCeilingFrags fragments of
// 1 KiB from frags; out gets each lane's sum of its 32 accumulator blocks
// (workgroups x 512 x 4 int32).
constexpr int kMfmaCeilingFrags = 24;
void launch_mfma_ceiling(const int8_t *frags, int32_t *out, int workgroups, int iters,
                         hipStream_t st);

void launch_sgd_requant(int8_t *qw, float *sw, const float *dw, int64_t N, int64_t K, float lr,
                        uint64_t seed, uint64_t step, float *bias, const float *db,
                        hipStream_t st);

// AdamW hyperparameters and the step constants derived from them on the host.
struct AdamConsts {
    float b1, b2, eps, a1, a2, c1, c2, decay;
};

// Row weight normalization: preparation and the SGD step (sgd.hip).
void launch_wn_init(const int8_t *q, const float *s, int64_t N, int64_t K, float *g, float *sw,
                    hipStream_t st);
void launch_wn_sgd_requant(int8_t *q, float *s, float *g, float *sw, const float *dw, int64_t N,
                           int64_t K, float lr, uint64_t seed, uint64_t step, float *bias,
                           const float *db, hipStream_t st);
void launch_adamw_requant(int8_t *qw, float *sw, const float *dw, float *m, float *v, int64_t N,
                          int64_t K, const AdamConsts &k, uint64_t seed, uint64_t step,
                          float *bias, const float *db, float *bm, float *bv, hipStream_t st);

// RMS norm with the residual's addition and INT8 rows as its output, and its
// backward pass (norm.hip).  part holds rmsnorm_bwd_parts(rows, cols) rows of
// cols floats.
void launch_rmsnorm_quant(const void *x, const void *res, bool bf16, int64_t rows, int64_t cols,
                          const float *gamma, float eps, int had, float cb, void *h, int8_t *q,
                          float *s, float *rstd, void *y, hipStream_t st);
int rmsnorm_bwd_parts(int64_t rows, int64_t cols);
void launch_rmsnorm_bwd(const void *dn, bool dn_bf16, const void *h, const void *dres, bool bf16,
                        const float *rstd, const float *gamma, int64_t rows, int64_t cols, void *dh,
                        float *dgamma, float *part, hipStream_t st);

// AdamW over the tensors of a device image (tensors.hpp, adamw.hip).
struct AdamTensorConsts {
    float b1, b2, eps, a1, a2, c1, c2, lr;
};
void launch_adamw_tensors(const void *image, int64_t count, int64_t chunks, const AdamTensorConsts &k,
                          uint64_t seed, uint64_t step, hipStream_t st);

// Low-rank adapters beside a projection (adapter.hip).  a [L, R, K] and b
// [L, N, R] are fp32 or bf16; ids [M] names each token's adapter.
constexpr int kMaxAdapters = 1023;
struct AdapterArgs {
    const void *a, *b;
    bool bf16;
    const float *scale;
    const int32_t *ids;
    int64_t M, N, K;
    int L, R;
};
// u = scale x^ A^T, with a workspace of adapter_fwd_bytes and kAdapterCountBytes of
// arrival counters (zero before and after); the result is u as bf16 terms, in the
// workspace.
constexpr size_t kAdapterCountBytes = 4096;
size_t adapter_fwd_bytes(int64_t M, int64_t R);
const uint16_t *launch_adapter_u(const AdapterArgs &g, const int8_t *qx, const float *sx, float *u,
                                 unsigned *count, void *ws, hipStream_t st);
void launch_adapter_group(const int32_t *ids, int64_t M, int L, int32_t *order, int32_t *start,
                          hipStream_t st);
// Backward, with a workspace of adapter_bwd_bytes: v = scale dY B (kept in
// the workspace; the result says where it and A's transpose lie, for the dX
// product), then both adapter gradients.
size_t adapter_bwd_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R);
AdapterEpilogue launch_adapter_bwd_v(const AdapterArgs &g, const void *dy, bool dy_bf16,
                                     const int32_t *start, float *da, float *db, unsigned *count,
                                     void *ws, hipStream_t st);
void launch_adapter_bwd_w(const AdapterArgs &g, const void *dy, bool dy_bf16, const int8_t *qx,
                          const float *sx, const float *u, const int32_t *order, float *da,
                          float *db, const AdapterTermArgs *dx, void *ws, hipStream_t st);

} // namespace qlin
