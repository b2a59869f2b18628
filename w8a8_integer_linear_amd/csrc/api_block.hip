// C-ABI entry points inside a feed-forward block: the products with activation, gate,
// residual and checkpoint, their backward, and the codes of a gradient whose scales
// are known.  As in api.hip, every check runs before the first launch.
#include "qlin.h"
#include "checks.hpp"
#include "launch.hpp"

namespace {

bool act_ok(int act) { return act >= QLIN_ACT_NONE && act <= QLIN_ACT_GELU_TANH; }

// Scales per row of a checkpoint.
int64_t ck_scales(int64_t F, bool gated)
{
    const int64_t per = (F + QLIN_CK_BLOCK - 1) / QLIN_CK_BLOCK;
    return gated ? 2 * per : per;
}

size_t fwd_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K > QLIN_MAX_CONTRACTION)
        return 0;
    return qlin::split_ws_bytes(qlin::act_split_plan(M, N, K));
}

// Both forward calls; N = 2 F with a gate.
int forward(const int8_t *qx, const float *sx, const int8_t *qw, const float *sw, const float *bias, int act,
            bool gated, const void *residual, int res_dtype, int64_t M, int64_t F, int64_t K, void *y,
            int y_dtype, int8_t *ck, float *ck_s, void *workspace, size_t ws_bytes, void *stream)
{
    if (!act_ok(act) || !dtype_ok(y_dtype) || (residual && !dtype_ok(res_dtype)) || !dim16(F))
        return QLIN_EINVAL;
    // (Past every limit, still a multiple of 16.)
    const int64_t N = gated ? 2 * (F < kMaxRows ? F : kMaxRows) : F;
    const int st = check_product(QLIN_OP_FWD, qx, qw, y, M, N, K);
    if (st == QLIN_EINVAL)
        return st;
    const bool any = M > 0;
    if (!array_ok(sx, any) || !array_ok(sw, any) || !opt_aligned(bias) || !opt_aligned(residual) ||
        !opt_aligned(ck) || !opt_aligned(ck_s) || (any && (ck != nullptr) != (ck_s != nullptr)))
        return QLIN_EINVAL;
    if (st != QLIN_OK || N > QLIN_MAX_BLOCK_ROWS)
        return QLIN_EUNSUPPORTED;
    if (!any)
        return QLIN_OK;
    const size_t need = fwd_ws_bytes(M, N, K);
    if (need && (!workspace || !aligned16(workspace) || ws_bytes < need))
        return QLIN_EINVAL;
    const int64_t ny = sat_mul(M, F, size_of(y_dtype)), nr = residual ? sat_mul(M, F, size_of(res_dtype)) : 0;
    // (The residual may be y itself.)
    const bool same = residual == y && nr == ny;
    const Range out[] = {{y, ny}, {ck, ck ? sat_mul(M, N) : 0}, {ck_s, ck ? sat_mul(M, ck_scales(F, gated), 4) : 0},
                         {workspace, (int64_t)need}};
    const Range in[] = {{qx, sat_mul(M, K)}, {qw, sat_mul(N, K)}, {sx, M * 4}, {sw, N * 4},
                        {bias, bias ? N * 4 : 0}, {residual, same ? 0 : nr}};
    if (clash(out, in))
        return QLIN_EINVAL;
    qlin::ProductArgs p{QLIN_OP_FWD, qx, qw, M, N, K, sx, sw, bias, y, false};
    if (need)
        p.split_ws = workspace;
    qlin::launch_product_act(p, {act, gated, F, y_dtype == QLIN_BF16, residual, res_dtype == QLIN_BF16, ck, ck_s},
                             as_stream(stream));
    return finish();
}

} // namespace

extern "C" {

size_t qlin_fwd_act_ws_bytes(int64_t M, int64_t N, int64_t K) { return fwd_ws_bytes(M, N, K); }

int qlin_fwd_act(const int8_t *qx, const float *sx, const int8_t *qw, const float *sw, const float *bias,
                 int act, const void *residual, int res_dtype, int64_t M, int64_t N, int64_t K, void *y,
                 int y_dtype, int8_t *ck, float *ck_s, void *workspace, size_t ws_bytes, void *stream)
{
    return forward(qx, sx, qw, sw, bias, act, false, residual, res_dtype, M, N, K, y, y_dtype, ck, ck_s,
                   workspace, ws_bytes, stream);
}

size_t qlin_fwd_gated_ws_bytes(int64_t M, int64_t F, int64_t K)
{
    return F < 0 || F > kMaxRows ? 0 : fwd_ws_bytes(M, 2 * F, K);
}

int qlin_fwd_gated(const int8_t *qx, const float *sx, const int8_t *qw, const float *sw, const float *bias,
                   int act, int64_t M, int64_t F, int64_t K, void *y, int y_dtype, int8_t *ck, float *ck_s,
                   void *workspace, size_t ws_bytes, void *stream)
{
    return forward(qx, sx, qw, sw, bias, act, true, nullptr, QLIN_F32, M, F, K, y, y_dtype, ck, ck_s,
                   workspace, ws_bytes, stream);
}

size_t qlin_act_bwd_ws_bytes(int64_t M, int64_t F, int gated)
{
    if (M < 0 || M > kMaxRows || !dim16(F) || sat_mul(F, gated ? 2 : 1) > QLIN_MAX_BLOCK_ROWS)
        return 0;
    return qlin::act_bwd_bytes(M, F, gated != 0);
}

int qlin_act_bwd(const void *dy, int dy_dtype, const int8_t *ck, const float *ck_s, int act, int gated,
                 const float *sw, const float *sx, int64_t M, int64_t F, void *dz, int dz_dtype, float *s1,
                 float *s2, float *db, void *workspace, size_t ws_bytes, void *stream)
{
    if (!act_ok(act) || (gated != 0 && gated != 1) || !dtype_ok(dy_dtype) || !dtype_ok(dz_dtype) || M < 0 ||
        !dim16(F))
        return QLIN_EINVAL;
    const bool any = M > 0;
    if (!array_ok(dy, any) || !array_ok(ck, any) || !array_ok(ck_s, any) || !array_ok(dz, any) ||
        !opt_aligned(sw) || !opt_aligned(sx) || !opt_aligned(s1) || !opt_aligned(s2) || !opt_aligned(db))
        return QLIN_EINVAL;
    // (Arrays of M elements may be null without rows.)
    if (any && ((sw != nullptr) != (s1 != nullptr) || (sx != nullptr) != (s2 != nullptr)))
        return QLIN_EINVAL;
    const int64_t N = sat_mul(F, gated ? 2 : 1);
    if (N > QLIN_MAX_BLOCK_ROWS || M > kMaxRows)
        return QLIN_EUNSUPPORTED;
    const size_t need = qlin_act_bwd_ws_bytes(M, F, gated);
    if (any && (!workspace || !aligned16(workspace) || ws_bytes < need))
        return QLIN_EINVAL;
    const int64_t nr = M * 4, nc = N * 4;
    const Range out[] = {{dz, sat_mul(M, N, size_of(dz_dtype))}, {s1, s1 ? nr : 0}, {s2, s2 ? nc : 0},
                         {db, db ? nc : 0}, {workspace, any ? (int64_t)need : 0}};
    const Range in[] = {{dy, sat_mul(M, F, size_of(dy_dtype))}, {ck, sat_mul(M, N)},
                        {ck_s, sat_mul(M, ck_scales(F, gated != 0), 4)}, {sw, sw ? nc : 0}, {sx, sx ? nr : 0}};
    if (clash(out, in))
        return QLIN_EINVAL;
    qlin::launch_act_bwd({dy, dy_dtype == QLIN_BF16, ck, ck_s, act, gated != 0, sw, sx, M, F, dz,
                          dz_dtype == QLIN_BF16, any ? s1 : nullptr, s2, db},
                         workspace, as_stream(stream));
    return finish();
}

int qlin_quantize_grad_scaled(const void *dy, int dtype, int64_t M, int64_t N, const float *sw, const float *sx,
                              const float *s1, const float *s2, int8_t *q1, int8_t *q2, void *stream)
{
    if (!dtype_ok(dtype) || M < 0 || !dim16(N))
        return QLIN_EINVAL;
    const bool any = M > 0;
    if (!array_ok(dy, any) || !array_ok(sw, any) || !array_ok(sx, any) || !array_ok(s1, any) ||
        !array_ok(s2, any) || !array_ok(q1, any) || !array_ok(q2, any))
        return QLIN_EINVAL;
    const int64_t n = sat_mul(M, N), nr = sat_mul(M, 4), nc = sat_mul(N, 4);
    const Range out[] = {{q1, n}, {q2, n}};
    const Range in[] = {{dy, sat_mul(M, N, size_of(dtype))}, {sw, nc}, {sx, nr}, {s1, nr}, {s2, nc}};
    if (clash(out, in))
        return QLIN_EINVAL;
    if (N > QLIN_MAX_ROW || M > 65535LL * 16)       // (grid.y stays below 65536)
        return QLIN_EUNSUPPORTED;
    if (!any)
        return QLIN_OK;
    qlin::launch_grad_codes(dy, dtype == QLIN_BF16, M, N, sw, sx, s1, s2, q1, q2, as_stream(stream));
    return finish();
}

} // extern "C"
