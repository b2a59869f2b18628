// C-ABI entry points around the projection: the norm, the adapters and the
// multi-tensor optimizer step.  As in api.hip, every check runs before the
// first launch.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "qlin.h"
#include "checks.hpp"
#include "launch.hpp"
#include "tensors.hpp"

namespace {

int64_t size_of(int dtype) { return dtype == QLIN_BF16 ? 2 : 4; }

// A byte range; [p, p + n).
struct Range {
    const void *p;
    int64_t n;
};

// Whether any of the written ranges meets another range of either list.
template <size_t W, size_t R>
bool clash(const Range (&written)[W], const Range (&read)[R])
{
    for (size_t i = 0; i < W; i++) {
        for (size_t j = i + 1; j < W; j++)
            if (overlap(written[i].p, written[i].n, written[j].p, written[j].n))
                return true;
        for (size_t j = 0; j < R; j++)
            if (overlap(written[i].p, written[i].n, read[j].p, read[j].n))
                return true;
    }
    return false;
}

// Like overlap, but the same array twice is allowed (an in-place call).
bool partly(const void *a, const void *b, int64_t n) { return a != b && overlap(a, n, b, n); }

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

bool adapter_shape_ok(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    return M >= 0 && M <= QLIN_MAX_ADAPTER_ROWS && dim16(N) && dim16(K) && N <= kMaxRows &&
           K <= kMaxRows && L >= 1 && L <= INT32_MAX && R >= 8 && R <= QLIN_MAX_RANK && R % 8 == 0;
}

// Whether the launches of a backward call hold its gradients: the preparation has
// a workgroup of 256 per 32 x 32 of A and B, the sums one per 1024 values, and a
// grid's dimension fewer than 2^32 threads.
bool gradients_fit(int64_t N, int64_t K, int64_t R)
{
    return (R + 31) / 32 * 32 * (N + K) <= QLIN_MAX_ADAPTER_SIZE;
}

int check_adapter(const void *a, const void *b, int w_dtype, const float *scale, const int32_t *ids,
                  int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    if (!dtype_ok(w_dtype) || L < 1 || R < 8 || R > QLIN_MAX_RANK || R % 8 != 0)
        return QLIN_EINVAL;
    if (!array_ok(a, true) || !array_ok(b, true) || !array_ok(scale, true) || !array_ok(ids, M > 0))
        return QLIN_EINVAL;
    if (M > QLIN_MAX_ADAPTER_ROWS || L > INT32_MAX || sat_mul(L, N, R) > ((int64_t)1 << 40) ||
        sat_mul(L, K, R) > ((int64_t)1 << 40))
        return QLIN_EUNSUPPORTED;
    return QLIN_OK;
}

} // namespace

extern "C" {

int qlin_rmsnorm_quant(const void *x, const void *residual, int dtype, int64_t rows, int64_t cols,
                       const float *gamma, float eps, int had_block, void *h, int8_t *q, float *s,
                       float *rstd, void *y, void *stream)
{
    if (!dtype_ok(dtype) || rows < 0 || !dim16(cols) || !(eps > 0.0f) || !isfinite(eps))
        return QLIN_EINVAL;
    const bool any = rows > 0;
    if (!array_ok(x, any) || !array_ok(q, any) || !array_ok(s, any) || !array_ok(rstd, any) ||
        !array_ok(gamma, true) || !opt_aligned(residual) || !opt_aligned(h) || !opt_aligned(y))
        return QLIN_EINVAL;
    if (any && (residual != nullptr) != (h != nullptr))
        return QLIN_EINVAL;
    if (had_block != 0 && !hadamard_block_ok(cols, had_block))
        return QLIN_EINVAL;
    const int64_t n = sat_mul(rows, cols), nx = sat_mul(rows, cols, size_of(dtype));
    if (h && (partly(h, x, nx) || partly(h, residual, nx)))
        return QLIN_EINVAL;
    const Range out[] = {{q, n}, {s, sat_mul(rows, 4)}, {rstd, sat_mul(rows, 4)}, {y, y ? sat_mul(n, 2) : 0}};
    const Range in[] = {{x, nx}, {residual, residual ? nx : 0}, {h, h ? nx : 0}, {gamma, sat_mul(cols, 4)}};
    if (any && (clash(out, in) || overlap(h, h ? nx : 0, gamma, sat_mul(cols, 4))))
        return QLIN_EINVAL;
    if (cols > QLIN_MAX_ROW || rows > kMaxRows)
        return QLIN_EUNSUPPORTED;
    if (!any)
        return QLIN_OK;
    qlin::launch_rmsnorm_quant(x, residual, dtype == QLIN_BF16, rows, cols, gamma, eps, had_block,
                               had_block ? hadamard_scale(had_block) : 1.0f, h, q, s, rstd, y,
                               as_stream(stream));
    return finish();
}

size_t qlin_rmsnorm_bwd_ws_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || rows > kMaxRows || !dim16(cols) || cols > QLIN_MAX_ROW)
        return 0;
    return (size_t)qlin::rmsnorm_bwd_parts(rows, cols) * (size_t)cols * 4;
}

int qlin_rmsnorm_bwd(const void *dn, int dn_dtype, const void *h, const void *dres, int dtype,
                     const float *rstd, const float *gamma, int64_t rows, int64_t cols, void *dh,
                     float *dgamma, void *workspace, size_t ws_bytes, void *stream)
{
    if (!dtype_ok(dn_dtype) || !dtype_ok(dtype) || rows < 0 || !dim16(cols))
        return QLIN_EINVAL;
    const bool any = rows > 0;
    if (!array_ok(dn, any) || !array_ok(h, any) || !opt_aligned(dres) || !array_ok(rstd, any) ||
        !array_ok(gamma, true) || !array_ok(dh, any) || !array_ok(dgamma, true) ||
        !array_ok(workspace, any))
        return QLIN_EINVAL;
    const int64_t n = sat_mul(rows, cols, size_of(dtype)), nd = sat_mul(rows, cols, size_of(dn_dtype));
    const int64_t nc = sat_mul(cols, 4);
    if (cols > QLIN_MAX_ROW || rows > kMaxRows)
        return QLIN_EUNSUPPORTED;
    const size_t need = qlin_rmsnorm_bwd_ws_bytes(rows, cols);
    if (ws_bytes < need)
        return QLIN_EINVAL;
    const Range out[] = {{dh, n}, {dgamma, nc}, {workspace, (int64_t)need}};
    const Range in[] = {{dn, nd}, {h, n}, {rstd, sat_mul(rows, 4)}, {gamma, nc}};
    const Range out2[] = {{dgamma, nc}, {workspace, (int64_t)need}};
    const Range in2[] = {{dres, dres ? n : 0}};
    if (any && (clash(out, in) || clash(out2, in2) || (dres && partly(dh, dres, n))))
        return QLIN_EINVAL;
    if (!any && overlap(dgamma, nc, gamma, nc))
        return QLIN_EINVAL;
    qlin::launch_rmsnorm_bwd(dn, dn_dtype == QLIN_BF16, h, dres, dtype == QLIN_BF16, rstd, gamma, rows,
                             cols, dh, dgamma, static_cast<float *>(workspace), as_stream(stream));
    return finish();
}

// Where the parts of an adapter call's workspace lie: both kinds of arrival
// counters first, at the same places for every call and shape (so that one
// workspace serves them all), then the product's sums, then the adapters' part.
struct AdapterWs {
    unsigned *count;
    char *product, *rest;
};
static size_t product_part(int op, int64_t M, int64_t N, int64_t K)
{
    const size_t n = qlin_product_ws_bytes(op, M, N, K);
    return qlin::kAdapterCountBytes + round256(n > qlin::kSplitCountBytes ? n : qlin::kSplitCountBytes);
}
static AdapterWs parts_of(void *workspace, int op, int64_t M, int64_t N, int64_t K)
{
    char *w = static_cast<char *>(workspace);
    return {static_cast<unsigned *>(workspace), w + qlin::kAdapterCountBytes, w + product_part(op, M, N, K)};
}

size_t qlin_adapter_fwd_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    if (!adapter_shape_ok(M, N, K, L, R) || K > QLIN_MAX_CONTRACTION)
        return 0;
    return product_part(QLIN_OP_FWD, M, N, K) + qlin::adapter_fwd_bytes(M, R);
}

int qlin_adapter_fwd(const int8_t *qx, const float *sx, const int8_t *qw, const float *sw,
                     const float *bias, const void *a, const void *b, int w_dtype,
                     const float *scale, const int32_t *ids, int64_t M, int64_t N, int64_t K,
                     int64_t L, int64_t R, float *u, float *y, void *workspace, size_t ws_bytes,
                     void *stream)
{
    int st = check_product(QLIN_OP_FWD, qx, qw, y, M, N, K);
    if (st == QLIN_EINVAL)
        return st;
    const int sa = check_adapter(a, b, w_dtype, scale, ids, M, N, K, L, R);
    if (sa == QLIN_EINVAL || !array_ok(u, M > 0) || !opt_aligned(bias) || !array_ok(sx, M > 0) ||
        !array_ok(sw, M > 0))
        return QLIN_EINVAL;
    if (st != QLIN_OK || sa != QLIN_OK)
        return QLIN_EUNSUPPORTED;
    if (M == 0)
        return QLIN_OK;
    const size_t need = qlin_adapter_fwd_ws_bytes(M, N, K, L, R);
    if (need && (!workspace || !aligned16(workspace) || ws_bytes < need))
        return QLIN_EINVAL;
    const int64_t e = size_of(w_dtype);
    const Range out[] = {{y, sat_mul(M, N, 4)}, {u, sat_mul(M, R, 4)}, {workspace, (int64_t)need}};
    const Range in[] = {{qx, M * K}, {qw, sat_mul(N, K)}, {sx, M * 4}, {sw, N * 4},
                        {bias, bias ? N * 4 : 0}, {a, L * R * K * e}, {b, L * R * N * e},
                        {scale, L * 4}, {ids, M * 4}};
    if (clash(out, in))
        return QLIN_EINVAL;
    const hipStream_t s = as_stream(stream);
    qlin::ProductArgs p{QLIN_OP_FWD, qx, qw, M, N, K, sx, sw, bias, y, false};
    const AdapterWs w = parts_of(workspace, QLIN_OP_FWD, M, N, K);
    if (qlin_product_ws_bytes(QLIN_OP_FWD, M, N, K))
        p.split_ws = w.product;
    const qlin::AdapterArgs g{a, b, w_dtype == QLIN_BF16, scale, ids, M, N, K, (int)L, (int)R};
    const uint16_t *terms = qlin::launch_adapter_u(g, qx, sx, u, w.count, w.rest, s);
    qlin::launch_product_adapter(p, {u, terms, b, ids, (int)L, (int)R, g.bf16}, s);
    return finish();
}

int qlin_adapter_group(const int32_t *ids, int64_t M, int64_t L, int32_t *order, int32_t *start,
                       void *stream)
{
    if (M < 0 || L < 1 || !array_ok(ids, M > 0) || !array_ok(order, M > 0) || !array_ok(start, true))
        return QLIN_EINVAL;
    if (M > QLIN_MAX_ADAPTER_ROWS || L > QLIN_MAX_ADAPTERS)
        return QLIN_EUNSUPPORTED;
    const Range out[] = {{order, M * 4}, {start, (L + 1) * 4}};
    const Range in[] = {{ids, M * 4}};
    if (clash(out, in))
        return QLIN_EINVAL;
    qlin::launch_adapter_group(ids, M, (int)L, order, start, as_stream(stream));
    return finish();
}

size_t qlin_adapter_bwd_ws_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    if (!adapter_shape_ok(M, N, K, L, R) || N > QLIN_MAX_CONTRACTION || L > QLIN_MAX_ADAPTERS ||
        !gradients_fit(N, K, R))
        return 0;
    return product_part(QLIN_OP_DX, M, N, K) + qlin::adapter_bwd_bytes(M, N, K, L, R);
}

int qlin_adapter_bwd(const void *dy, int dy_dtype, const int8_t *qg1, const float *sg1,
                     const int8_t *qw, const int8_t *qx, const float *sx, const float *u,
                     const void *a, const void *b, int w_dtype, const float *scale,
                     const int32_t *ids, const int32_t *order, const int32_t *start, int64_t M,
                     int64_t N, int64_t K, int64_t L, int64_t R, int had_block, float *dx,
                     float *da, float *db, void *workspace, size_t ws_bytes, void *stream)
{
    const bool any = M > 0;
    if (!dtype_ok(dy_dtype) || M < 0 || !dim16(N) || !dim16(K))
        return QLIN_EINVAL;
    int st = dx ? check_product(QLIN_OP_DX, qg1, qw, dx, M, N, K)
                : (N > QLIN_MAX_CONTRACTION || K > kMaxRows ? QLIN_EUNSUPPORTED : QLIN_OK);
    if (st == QLIN_EINVAL)
        return st;
    if (had_block != 0 && !hadamard_block_ok(K, had_block))
        return QLIN_EINVAL;
    const int sa = check_adapter(a, b, w_dtype, scale, ids, M, N, K, L, R);
    if (sa == QLIN_EINVAL || !array_ok(dy, any) || !array_ok(qx, any) || !array_ok(sx, any) ||
        !array_ok(u, any) || !array_ok(order, any) || !array_ok(start, true) || !array_ok(da, true) ||
        !array_ok(db, true) || (dx && !array_ok(sg1, any)))
        return QLIN_EINVAL;
    if (st != QLIN_OK || sa != QLIN_OK || L > QLIN_MAX_ADAPTERS || !gradients_fit(N, K, R))
        return QLIN_EUNSUPPORTED;
    const size_t need = qlin_adapter_bwd_ws_bytes(M, N, K, L, R);
    if (!workspace || !aligned16(workspace) || ws_bytes < need)
        return QLIN_EINVAL;
    const int64_t e = size_of(w_dtype);
    const Range out[] = {{dx, dx ? sat_mul(M, K, 4) : 0}, {da, L * R * K * 4}, {db, L * R * N * 4},
                         {workspace, (int64_t)need}};
    const Range in[] = {{dy, sat_mul(M, N, size_of(dy_dtype))}, {qg1, dx ? M * N : 0},
                        {sg1, dx ? M * 4 : 0}, {qw, dx ? sat_mul(N, K) : 0}, {qx, M * K},
                        {sx, M * 4}, {u, M * R * 4}, {a, L * R * K * e}, {b, L * R * N * e},
                        {scale, L * 4}, {ids, M * 4}, {order, M * 4}, {start, (L + 1) * 4}};
    if (clash(out, in))
        return QLIN_EINVAL;
    const hipStream_t s = as_stream(stream);
    const AdapterWs w = parts_of(workspace, QLIN_OP_DX, M, N, K);
    const qlin::AdapterArgs g{a, b, w_dtype == QLIN_BF16, scale, ids, M, N, K, (int)L, (int)R};
    const qlin::AdapterEpilogue va =
        qlin::launch_adapter_bwd_v(g, dy, dy_dtype == QLIN_BF16, start, da, db, w.count, w.rest, s);
    const bool bf = dy_dtype == QLIN_BF16;
    if (!any || !dx) {
        qlin::launch_adapter_bwd_w(g, dy, bf, qx, sx, u, order, da, db, nullptr, w.rest, s);
        return finish();
    }
    qlin::ProductArgs p{QLIN_OP_DX, qg1, qw, M, N, K, sg1, nullptr, nullptr, dx, false};
    if (qlin_product_ws_bytes(QLIN_OP_DX, M, N, K))
        p.split_ws = w.product;
    const float cb = had_block ? hadamard_scale(had_block) : 1.0f;
    if (qlin::adapter_term_apart(M, K)) {
        // The product, then its term with the gradients.
        qlin::launch_product(p, s);
        const qlin::AdapterTermArgs term{va, M, K, dx, had_block >= 2 && had_block <= 128 ? had_block : 0, cb};
        qlin::launch_adapter_bwd_w(g, dy, bf, qx, sx, u, order, da, db, &term, w.rest, s);
    } else {
        // The gradients come first: they read dY again, while the product with B
        // has just left what fits of it in the infinity cache.
        qlin::launch_adapter_bwd_w(g, dy, bf, qx, sx, u, order, da, db, nullptr, w.rest, s);
        p.had = had_block;
        p.had_scale = cb;
        qlin::launch_product_adapter(p, va, s);
    }
    if (had_block > 128)
        qlin::launch_hadamard(dx, false, M, K, had_block, cb, dx, s);
    return finish();
}

// ------------------------------------------------------ multi-tensor AdamW

static int64_t chunks_of(int64_t numel)
{
    return numel / qlin::kTensorChunk + (numel % qlin::kTensorChunk != 0);
}

int64_t qlin_adamw_tensors_chunks(const qlin_tensor *tensors, int64_t count)
{
    int64_t n = 0;
    if (!tensors)
        return 0;
    for (int64_t i = 0; i < count; i++)
        if (tensors[i].numel > 0 && __builtin_add_overflow(n, chunks_of(tensors[i].numel), &n))
            return INT64_MAX;
    return n;
}

size_t qlin_adamw_tensors_plan_bytes(const qlin_tensor *tensors, int64_t count)
{
    const int64_t n = qlin_adamw_tensors_chunks(tensors, count);
    if (count <= 0 || count > INT32_MAX || n > INT32_MAX)
        return 0;
    return (size_t)count * sizeof(qlin::TensorEntry) + (size_t)n * 4;
}

int qlin_adamw_tensors_plan(const qlin_tensor *tensors, int64_t count, void *image, size_t image_bytes)
{
    if (count < 0 || (count > 0 && !tensors))
        return QLIN_EINVAL;
    std::vector<std::pair<uintptr_t, uintptr_t>> written, read;
    try {
        for (int64_t i = 0; i < count; i++) {
            const qlin_tensor &t = tensors[i];
            const bool any = t.numel > 0, eight = t.state_bits == 8;
            if (t.numel < 0 || !dtype_ok(t.p_dtype) || !dtype_ok(t.g_dtype) ||
                (t.state_bits != 8 && t.state_bits != 32) || !isfinite(t.weight_decay) ||
                t.weight_decay < 0.0f || t.index0 < 0 || t.index0 % 8 != 0)
                return QLIN_EINVAL;
            if (!array_ok(t.p, any) || !array_ok(t.g, any) || !array_ok(t.m, any) || !array_ok(t.v, any))
                return QLIN_EINVAL;
            if (any && (eight != (t.m_scale != nullptr) || eight != (t.v_scale != nullptr)))
                return QLIN_EINVAL;
            // (Scales are read and written one at a time: four-byte aligned.)
            if (((uintptr_t)t.m_scale | (uintptr_t)t.v_scale) & 3)
                return QLIN_EINVAL;
            if (t.numel > ((int64_t)1 << 42) || t.index0 > ((int64_t)1 << 62))
                return QLIN_EUNSUPPORTED;
            if (!any)
                continue;
            auto range = [](std::vector<std::pair<uintptr_t, uintptr_t>> &to, const void *p, int64_t n) {
                const uintptr_t b = (uintptr_t)p;
                to.emplace_back(b, (uint64_t)n > UINTPTR_MAX - b ? UINTPTR_MAX : b + (uintptr_t)n);
            };
            const int64_t blocks = (t.numel + qlin::kStateBlock - 1) / qlin::kStateBlock;
            range(written, t.p, t.numel * size_of(t.p_dtype));
            range(written, t.m, t.numel * (eight ? 1 : 4));
            range(written, t.v, t.numel * (eight ? 1 : 4));
            if (eight) {
                range(written, t.m_scale, blocks * 4);
                range(written, t.v_scale, blocks * 4);
            }
            range(read, t.g, t.numel * size_of(t.g_dtype));
        }
        // No written range meets another written one, nor a gradient.
        std::sort(written.begin(), written.end());
        for (size_t i = 1; i < written.size(); i++)
            if (written[i].first < written[i - 1].second)
                return QLIN_EINVAL;
        for (const auto &r : read) {
            auto it = std::upper_bound(written.begin(), written.end(),
                                       std::make_pair(r.first, UINTPTR_MAX));
            if ((it != written.end() && it->first < r.second) ||
                (it != written.begin() && std::prev(it)->second > r.first))
                return QLIN_EINVAL;
        }
    } catch (...) {     // the host's memory ran out
        return QLIN_EDEVICE;
    }
    const int64_t chunks = qlin_adamw_tensors_chunks(tensors, count);
    if (count > INT32_MAX || chunks > INT32_MAX)
        return QLIN_EUNSUPPORTED;
    if (count == 0)
        return QLIN_OK;
    const size_t need = qlin_adamw_tensors_plan_bytes(tensors, count);
    if (!image || image_bytes < need)
        return QLIN_EINVAL;
    char *at = static_cast<char *>(image), *map = at + count * sizeof(qlin::TensorEntry);
    int64_t chunk = 0;
    for (int64_t i = 0; i < count; i++) {
        const qlin_tensor &t = tensors[i];
        qlin::TensorEntry e;
        memset(&e, 0, sizeof e);
        e.p = t.p;
        e.g = t.g;
        e.m = t.m;
        e.v = t.v;
        e.ms = t.m_scale;
        e.vs = t.v_scale;
        e.numel = t.numel;
        e.index0 = t.index0;
        e.chunk0 = chunk;
        e.weight_decay = t.weight_decay;
        e.flags = (t.p_dtype == QLIN_BF16 ? qlin::kParamBf16 : 0) |
                  (t.g_dtype == QLIN_BF16 ? qlin::kGradBf16 : 0) |
                  (t.state_bits == 8 ? qlin::kState8 : 0);
        memcpy(at + i * sizeof e, &e, sizeof e);
        const int32_t id = (int32_t)i;
        for (int64_t c = chunks_of(t.numel); c > 0; c--, chunk++)
            memcpy(map + chunk * 4, &id, 4);
    }
    return QLIN_OK;
}

int qlin_adamw_tensors(const void *image, int64_t count, int64_t chunks, double lr, double beta1,
                       double beta2, double eps, uint64_t seed, uint64_t step, void *stream)
{
    if (count < 0 || chunks < 0 || step < 1 || !array_ok(image, chunks > 0) || (chunks > 0 && count == 0))
        return QLIN_EINVAL;
    if (!isfinite(lr) || !isfinite(eps) || !(eps > 0.0) || !((float)eps > 0.0f) ||
        !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
        return QLIN_EINVAL;
    if (count > INT32_MAX || chunks > INT32_MAX || step >> 63)
        return QLIN_EUNSUPPORTED;
    if (chunks == 0)
        return QLIN_OK;
    // Step constants, each computed in double and rounded once.  The step's quotient
    // has both its sides times 2^24 (c1 and c2, eps): the reciprocal instruction takes
    // a subnormal denominator for zero, and an element that never had a gradient would
    // get 0 / 0 where eps is one.
    const double t = (double)step, up = 0x1p24;
    qlin::AdamTensorConsts k;
    k.b1 = (float)beta1;
    k.b2 = (float)beta2;
    k.eps = (float)(eps * up);
    k.a1 = (float)(1.0 - beta1);
    k.a2 = (float)(1.0 - beta2);
    k.c1 = (float)(lr * up / (1.0 - pow(beta1, t)));
    k.c2 = (float)(up / sqrt(1.0 - pow(beta2, t)));
    k.lr = (float)lr;
    qlin::launch_adamw_tensors(image, count, chunks, k, seed, step, as_stream(stream));
    return finish();
}

} // extern "C"
