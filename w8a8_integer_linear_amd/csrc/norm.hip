// RMS norm with the residual's addition in front and the INT8 row quantizer
// behind it, and its backward pass.
//
// Forward, one row: h = rnd(x + residual) (in the stream's own type), rstd =
// 1 / sqrt(mean(h^2) + eps), n = (h * rstd) * gamma, g = rotate(n), s = max|g|
// / 127, q = rne(g / s).  A row's values stay in registers from the loads to
// the codes, so x and the residual are read once and h and q written once (above
// 32768 columns a lane has 64 of them or more and some go through scratch memory:
// up to 46 registers' worth, above 65536 columns 172 to 692); the row's two
// reductions (the sum of squares, the absmax) run across lanes.
// HBM traffic bounds it, except for a few rows, where the launch does: 12000 rows
// of 5376 in fp32 with a residual and the codes' values as bf16 beside them, 968
// MB, take 174 us (5.6 TB/s); 3 rows of 4096 take 3.4 us in the kernel and 5.6 us
// as a call.  Long rows, 64 M elements in bf16 with a residual: 5.5 TB/s up to 16384
// columns, 4.2 at 65536, 1.3 at 131072 (the scratch memory's traffic).  Short ones
// leave lanes without columns: 120000 rows of 512 take 261 us, 1.7 TB/s, as long as
// as many rows of 128.
//
// Backward, one row, with xh = h * rstd and g = dn * gamma: dh = dres + rstd
// (g - xh mean(g xh)), and dgamma += dn * xh per column.  A workgroup walks
// rows and keeps its columns' dgamma sums in registers; the workgroups'
// partial sums are added in a fixed order by a second kernel, so no result
// depends on the order of arrival.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "lowp.hpp"

namespace qlin {

namespace {

constexpr float kInf = __builtin_inff();

// Reduction over the workgroup's WPR waves, which share a row; every thread gets
// the result.  red holds one float per wave and is written again only after the
// next barrier that all its readers have passed (two arrays take turns for
// consecutive reductions).
template <int WPR, typename Op>
__device__ __forceinline__ float row_reduce(float v, float *red, Op op)
{
    v = wave_all(v, op);
    const int w = threadIdx.x / kWave;
    if (__lane_id() == 0)
        red[w] = v;
    lds_barrier();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WPR; i++)
        v = op(v, red[i]);
    return v;
}

// Stores of what nothing reads soon (h, y): cached, they would push the codes,
// which the products read next, out of the infinity cache.
template <typename V> __device__ __forceinline__ void store_once(void *p, V v)
{
    __builtin_nontemporal_store(v, static_cast<V *>(p));
}

struct NormArgs {
    const void *x, *res;
    int64_t rows, cols;
    const float *gamma;
    float eps;
    int had;
    float cb;
    void *h;            // null: no residual, the norm's input is x
    int8_t *q;
    float *s, *rstd;
    uint16_t *y;        // bf16 values of the codes, or null
};

// One row per workgroup of WPR waves, J chunks of eight elements per lane.
template <bool BF16, int WPR, int J, int HAD>
__global__ __launch_bounds__(WPR *kWave) void rmsnorm_quant_kernel(NormArgs a)
{
    constexpr int kThreads = WPR * kWave;
    __shared__ float red[2][WPR];
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int64_t nch = a.cols / 8, base = row * a.cols;
    auto chunk = [&](int j) {
        const int64_t c = t + (int64_t)j * kThreads;
        if constexpr (HAD > 0)
            return had_chunk<HAD>(c);
        else
            return c;
    };
    // Loads past the row's end read its last chunk; their values are dropped.
    Raw8<BF16> xr[J], rr[J];
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int64_t c = chunk(j), cc = c < nch ? c : nch - 1;
        xr[j] = load_raw8<BF16>(a.x, base + cc * 8);
    }
    if (a.res) {
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int64_t c = chunk(j), cc = c < nch ? c : nch - 1;
            rr[j] = load_raw8<BF16>(a.res, base + cc * 8);
        }
    }
    // gamma is loaded before h is stored: a load's wait includes the stores
    // issued before it.  (Rows of 1024 threads have no registers for it.)
    constexpr bool kEarly = WPR <= 4;
    Raw8<false> gr[kEarly ? J : 1];
    auto gamma_at = [&](int j) {
        const int64_t c = chunk(j);
        return load_raw8<false>(a.gamma, (c < nch ? c : nch - 1) * 8);
    };
    if constexpr (kEarly) {
#pragma unroll
        for (int j = 0; j < J; j++)
            gr[j] = gamma_at(j);
        __builtin_amdgcn_sched_barrier(0);
    }
    float v[J][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int64_t c = chunk(j);
        const bool ok = c < nch;
        unpack8<BF16>(xr[j], v[j]);
        if (a.res) {
            float r[8];
            unpack8<BF16>(rr[j], r);
#pragma unroll
            for (int e = 0; e < 8; e++)
                v[j][e] = v[j][e] + r[e];
            if constexpr (BF16) {
                // The norm is of the stream as it is stored, so that the
                // backward pass, which reads h, sees the same values.
                const i32x4 w = pack_bf16x8(v[j]);
                if (ok)
                    store_once(static_cast<uint16_t *>(a.h) + base + c * 8, w);
                unpack8<true>(Raw8<true>{w}, v[j]);
            } else if (ok) {
                store8(static_cast<float *>(a.h), base + c * 8, v[j]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            v[j][e] = ok ? v[j][e] : 0.0f;
            ss = __builtin_fmaf(v[j][e], v[j][e], ss);
        }
    }
    ss = row_reduce<WPR>(ss, red[0], [](float p, float q) { return p + q; });
    const float rstd = 1.0f / __builtin_sqrtf(ss / (float)a.cols + a.eps);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < J; j++) {
        float gm[8];
        unpack8<false>(kEarly ? gr[kEarly ? j : 0] : gamma_at(j), gm);
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[j][e] = (v[j][e] * rstd) * gm[e];
        if constexpr (HAD > 0)
            fwht8_fixed<HAD, false>(v[j], a.cb);
        else if constexpr (HAD < 0)
            fwht8_lanes(v[j], a.had, a.cb);
        // (Chunks past the end hold zeros, also after the rotation: a block is
        // past the end as a whole.)
#pragma unroll
        for (int e = 0; e < 8; e++)
            amax = max_nan(amax, __builtin_fabsf(v[j][e]));
    }
    amax = row_reduce<WPR>(amax, red[1], [](float p, float q) { return max_nan(p, q); });
    float sc = amax / 127.0f;
    // A row with an infinity or a NaN has no codes: its scale is NaN, so that
    // whatever is computed from it is NaN too, and its codes are zeros.  (The
    // sum of squares is checked by itself: an infinite one leaves rstd 0.)
    const bool bad = !(amax < kInf) || !(ss < kInf);
    if (bad)
        sc = __builtin_nanf("");
    if (t == 0) {
        a.s[row] = sc;
        a.rstd[row] = rstd;
    }
    const bool zero = bad || amax == 0.0f;
    const bool subnormal = !zero && sc < 0x1p-126f;
    const float inv = recip_refined(sc);
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int64_t c = chunk(j);
        i32x2 out;
        if (zero) {
            out = i32x2{0, 0};
        } else if (subnormal) {
            float r[8];
#pragma unroll
            for (int e = 0; e < 8; e++)
                r[e] = quant_code_exact(v[j][e], sc);
            out[0] = (int)pack4(r[0], r[1], r[2], r[3]);
            out[1] = (int)pack4(r[4], r[5], r[6], r[7]);
        } else {
            out = quant8(v[j], sc, inv);
        }
        if (c < nch) {
            *reinterpret_cast<i32x2 *>(a.q + base + c * 8) = out;
            if (a.y) {
                float f[8];
                codes_to_float(out, f);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    f[e] = f[e] * sc;
                store_once(a.y + base + c * 8, pack_bf16x8(f));
            }
        }
    }
}

template <bool BF16, int WPR, int J, int HAD>
void run_norm(const NormArgs &a, hipStream_t st)
{
    hipLaunchKernelGGL((rmsnorm_quant_kernel<BF16, WPR, J, HAD>), dim3((unsigned)a.rows),
                       dim3(WPR * kWave), 0, st, a);
}

template <bool BF16, int HAD>
void run_norm_h(const NormArgs &a, hipStream_t st)
{
    const int64_t nch = a.cols / 8;
    const int64_t j4 = (nch + 255) / 256;
    if (j4 <= 1)
        return run_norm<BF16, 4, 1, HAD>(a, st);
    if (j4 <= 2)
        return run_norm<BF16, 4, 2, HAD>(a, st);
    if (j4 <= 3)
        return run_norm<BF16, 4, 3, HAD>(a, st);
    if (j4 <= 4)
        return run_norm<BF16, 4, 4, HAD>(a, st);
    if (j4 <= 8)
        return run_norm<BF16, 4, 8, HAD>(a, st);
    const int64_t j16 = (nch + 1023) / 1024;
    if (j16 <= 4)
        return run_norm<BF16, 16, 4, HAD>(a, st);
    if (j16 <= 8)
        return run_norm<BF16, 16, 8, HAD>(a, st);
    return run_norm<BF16, 16, 16, HAD>(a, st);
}

template <bool BF16>
void run_norm_dt(const NormArgs &a, hipStream_t st)
{
    if (a.had == 0)
        run_norm_h<BF16, 0>(a, st);
    else if (a.had == 128)
        run_norm_h<BF16, 128>(a, st);
    else
        run_norm_h<BF16, -1>(a, st);
}

// Rows of one launch with up to 1024 threads each: a grid's dimension holds fewer
// than 2^32 threads (a larger one starts only what is left of it modulo 2^32, and
// reports no error).
constexpr int64_t kLaunchRows = (int64_t)1 << 21;

// --------------------------------------------------------------- backward

struct NormBwdArgs {
    const void *dn, *h, *dres;
    const float *rstd, *gamma;
    int64_t rows, cols;
    void *dh;
    float *dgamma, *part;       // part: [grid, cols] partial column sums
};

// One row at a time over 256 threads, J chunks per lane, the next row's loads in
// flight during the current one's reduction and stores (12000 x 5376, dn in fp32
// and the rest in bf16: 135 -> 119 us, 5.4 TB/s).
template <bool DNBF, bool BF16, int J>
__global__ __launch_bounds__(256, 2) void rmsnorm_bwd_kernel(NormBwdArgs a)
{
    __shared__ float red[2][4];
    const int t = threadIdx.x;
    const int64_t nch = a.cols / 8;
    float gm[J][8], dg[J][8];
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int64_t c = t + (int64_t)j * 256, cc = c < nch ? c : nch - 1;
        load8<false>(a.gamma, cc * 8, gm[j]);
#pragma unroll
        for (int e = 0; e < 8; e++)
            dg[j][e] = 0.0f;
    }
    Raw8<DNBF> dr[J];
    Raw8<BF16> hr[J], rr[J];
    float next_rstd = 0.0f;
    auto load = [&](int64_t row) {
        const int64_t base = row * a.cols;
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int64_t c = t + (int64_t)j * 256, cc = c < nch ? c : nch - 1;
            dr[j] = load_raw8<DNBF>(a.dn, base + cc * 8);
            hr[j] = load_raw8<BF16>(a.h, base + cc * 8);
        }
        next_rstd = a.rstd[row];
    };
    auto load_res = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int64_t c = t + (int64_t)j * 256, cc = c < nch ? c : nch - 1;
            rr[j] = load_raw8<BF16>(a.dres, row * a.cols + cc * 8);
        }
    };
    load(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const int64_t base = row * a.cols;
        if (a.dres)
            load_res(row);
        const float rstd = next_rstd;
        float xh[J][8], g[J][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < J; j++) {
            const bool ok = t + (int64_t)j * 256 < nch;
            unpack8<BF16>(hr[j], xh[j]);
            unpack8<DNBF>(dr[j], g[j]);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                xh[j][e] = xh[j][e] * rstd;
                dg[j][e] = __builtin_fmaf(g[j][e], xh[j][e], dg[j][e]);
                g[j][e] = g[j][e] * gm[j][e];
                dot = ok ? __builtin_fmaf(g[j][e], xh[j][e], dot) : dot;
            }
        }
        // The next row's loads are in flight from here on.
        load(row + gridDim.x < a.rows ? row + gridDim.x : row);
        __builtin_amdgcn_sched_barrier(0);
        dot = row_reduce<4>(dot, red[turn], [](float p, float q) { return p + q; });
        const float mean = dot / (float)a.cols;
#pragma unroll
        for (int j = 0; j < J; j++) {
            const int64_t c = t + (int64_t)j * 256;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; e++)
                o[e] = rstd * __builtin_fmaf(-mean, xh[j][e], g[j][e]);
            if (a.dres) {
                float r[8];
                unpack8<BF16>(rr[j], r);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    o[e] = o[e] + r[e];
            }
            if (c < nch) {
                if constexpr (BF16)
                    store_once(static_cast<uint16_t *>(a.dh) + base + c * 8, pack_bf16x8(o));
                else
                    store8(static_cast<float *>(a.dh), base + c * 8, o);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < J; j++) {
        const int64_t c = t + (int64_t)j * 256;
        if (c < nch)
            store8(a.part, (int64_t)blockIdx.x * a.cols + c * 8, dg[j]);
    }
}

// Rows too long for the kernel above: each row is read twice (its dot
// product, then dh), and the column sums are a pass of their own (64 M elements, dn
// in fp32 and the rest in bf16: 12288 columns 211 us, 3.0 TB/s of what a single pass
// would move; 131072 columns 276 us).  Workgroup i has row r0 + i.
template <bool DNBF, bool BF16>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_long_kernel(NormBwdArgs a, int64_t r0)
{
    __shared__ float red[16];
    const int64_t nch = a.cols / 8, row = r0 + blockIdx.x, base = row * a.cols;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int64_t c = threadIdx.x; c < nch; c += 1024) {
        float x[8], g[8], gm[8];
        load8<BF16>(a.h, base + c * 8, x);
        load8<DNBF>(a.dn, base + c * 8, g);
        load8<false>(a.gamma, c * 8, gm);
#pragma unroll
        for (int e = 0; e < 8; e++)
            dot = __builtin_fmaf(g[e] * gm[e], x[e] * rstd, dot);
    }
    dot = row_reduce<16>(dot, red, [](float p, float q) { return p + q; });
    const float mean = dot / (float)a.cols;
    for (int64_t c = threadIdx.x; c < nch; c += 1024) {
        float x[8], g[8], gm[8], o[8];
        load8<BF16>(a.h, base + c * 8, x);
        load8<DNBF>(a.dn, base + c * 8, g);
        load8<false>(a.gamma, c * 8, gm);
#pragma unroll
        for (int e = 0; e < 8; e++)
            o[e] = rstd * __builtin_fmaf(-mean, x[e] * rstd, g[e] * gm[e]);
        if (a.dres) {
            float r[8];
            load8<BF16>(a.dres, base + c * 8, r);
#pragma unroll
            for (int e = 0; e < 8; e++)
                o[e] = o[e] + r[e];
        }
        if constexpr (BF16)
            *reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(a.dh) + base + c * 8) = pack_bf16x8(o);
        else
            store8(static_cast<float *>(a.dh), base + c * 8, o);
    }
}

// Column sums of dn * h * rstd over every gridDim.y-th row, into part.
template <bool DNBF, bool BF16>
__global__ __launch_bounds__(256) void rmsnorm_dgamma_kernel(NormBwdArgs a)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols / 8)
        return;
    float dg[8];
#pragma unroll
    for (int e = 0; e < 8; e++)
        dg[e] = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        float x[8], g[8];
        load8<BF16>(a.h, row * a.cols + c * 8, x);
        load8<DNBF>(a.dn, row * a.cols + c * 8, g);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; e++)
            dg[e] = __builtin_fmaf(g[e], x[e] * rstd, dg[e]);
    }
    store8(a.part, (int64_t)blockIdx.y * a.cols + c * 8, dg);
}

// dgamma = the column sums of part's n rows: 64 columns per workgroup, 16
// row lanes, added in a fixed order.
__global__ __launch_bounds__(1024) void rmsnorm_dgamma_sum_kernel(const float *__restrict__ part, int n,
                                                                  int64_t cols,
                                                                  float *__restrict__ dgamma)
{
    __shared__ float red[16][64];
    const int lc = threadIdx.x % 64, lr = threadIdx.x / 64;
    const int64_t c = (int64_t)blockIdx.x * 64 + lc;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int r = lr; r < n; r += 16)
            s = s + part[(int64_t)r * cols + c];
    }
    red[lr][lc] = s;
    __syncthreads();
    if (lr == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 16; i++)
            s = s + red[i][lc];
        dgamma[c] = s;
    }
}

// Longest row of the one-pass kernel.
constexpr int64_t kOnePassCols = 256 * 8 * 4;
// Workgroups that walk the rows, each with its own partial column sums.  Two per
// compute unit keep enough loads in flight (12000 rows of 2048 columns: 50 us
// with 512 workgroups, 56 us with 1536, whose partial sums are three times as
// many), except for rows so short that half of the lanes have no columns (30000
// rows of 1024: 87 us and 63 us).
constexpr int bwd_grid(int64_t cols) { return cols <= 1024 ? 1536 : 512; }

template <bool DNBF, bool BF16>
void run_bwd(const NormBwdArgs &a, int n, hipStream_t st)
{
    if (a.cols <= kOnePassCols) {
        const dim3 grid((unsigned)n), block(256);
        switch ((a.cols / 8 + 255) / 256) {
        case 1: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DNBF, BF16, 1>), grid, block, 0, st, a); break;
        case 2: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DNBF, BF16, 2>), grid, block, 0, st, a); break;
        case 3: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DNBF, BF16, 3>), grid, block, 0, st, a); break;
        default: hipLaunchKernelGGL((rmsnorm_bwd_kernel<DNBF, BF16, 4>), grid, block, 0, st, a);
        }
        return;
    }
    for (int64_t r0 = 0; r0 < a.rows; r0 += kLaunchRows) {
        const int64_t rows = a.rows - r0 < kLaunchRows ? a.rows - r0 : kLaunchRows;
        hipLaunchKernelGGL((rmsnorm_bwd_long_kernel<DNBF, BF16>), dim3((unsigned)rows), dim3(1024), 0, st,
                           a, r0);
    }
    hipLaunchKernelGGL((rmsnorm_dgamma_kernel<DNBF, BF16>),
                       dim3((unsigned)((a.cols / 8 + 255) / 256), (unsigned)n), dim3(256), 0, st, a);
}

} // namespace

void launch_rmsnorm_quant(const void *x, const void *res, bool bf16, int64_t rows, int64_t cols,
                          const float *gamma, float eps, int had, float cb, void *h, int8_t *q,
                          float *s, float *rstd, void *y, hipStream_t st)
{
    const int64_t size = bf16 ? 2 : 4;
    auto from = [](auto *p, int64_t byte) {
        return p ? (decltype(p))((uintptr_t)p + (uintptr_t)byte) : p;
    };
    for (int64_t r0 = 0; r0 < rows; r0 += kLaunchRows) {
        const int64_t n = rows - r0 < kLaunchRows ? rows - r0 : kLaunchRows, at = r0 * cols;
        const NormArgs a{from(x, at * size), from(res, at * size), n, cols, gamma, eps, had, cb,
                         from(h, at * size), q + at, s + r0, rstd + r0,
                         static_cast<uint16_t *>(from(y, at * 2))};
        if (bf16)
            run_norm_dt<true>(a, st);
        else
            run_norm_dt<false>(a, st);
    }
}

// Rows of partial column sums that a backward call writes.
int rmsnorm_bwd_parts(int64_t rows, int64_t cols)
{
    const int64_t most = cols <= kOnePassCols ? bwd_grid(cols) : 64;
    return (int)(rows < most ? rows : most);
}

void launch_rmsnorm_bwd(const void *dn, bool dn_bf16, const void *h, const void *dres, bool bf16,
                        const float *rstd, const float *gamma, int64_t rows, int64_t cols, void *dh,
                        float *dgamma, float *part, hipStream_t st)
{
    const NormBwdArgs a{dn, h, dres, rstd, gamma, rows, cols, dh, dgamma, part};
    const int n = rmsnorm_bwd_parts(rows, cols);
    if (rows > 0) {
        if (dn_bf16)
            bf16 ? run_bwd<true, true>(a, n, st) : run_bwd<true, false>(a, n, st);
        else
            bf16 ? run_bwd<false, true>(a, n, st) : run_bwd<false, false>(a, n, st);
    }
    hipLaunchKernelGGL(rmsnorm_dgamma_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st,
                       part, n, cols, dgamma);
}

} // namespace qlin
