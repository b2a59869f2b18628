// Backward of a feed-forward block's activation and gate from the 8-bit checkpoint of
// their input, up to the scales of the gradient's two quantizations: one pass over
// dy and the checkpoint that writes dz and leaves row maxima, column maxima and
// column sums as partials, and a small launch that reduces them.
#include <type_traits>

#include "act.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "lowp.hpp"

namespace qlin {

namespace {

constexpr int kCols = 512;      // outputs of a wave's window: eight per lane
constexpr int kWaves = 4;       // of a workgroup, one window, other rows
constexpr int kBatch = 2;       // rows a lane loads before it uses any of them
constexpr int kGroups = 4096;   // workgroups aimed at

struct Args {
    ActBackward a;
    int64_t N;                  // F, or 2 F with a gate
    int64_t per, all;           // checkpoint scales of a half and of a row
    float *rowpart;             // [windows, M]
    float *colpart;             // [2 groups, N]: maxima, then sums, of a row group
};

// Eight INT8 codes times a scale, each product rounded once: a code is taken as the
// unsigned byte c + 128, which one instruction converts, and 128 s is taken off in a
// fused multiply-add.  (A wave that meets a scale of 2^121 or more, where 128 s is past
// fp32, takes the codes themselves: z from 3.37e38 on have such a scale.  An infinite
// scale's codes say nothing of its block, which is NaN: s - s.)
__device__ __forceinline__ void codes_times(i32x2 q, float s, float v[8])
{
    if (__ballot(!(s < 0x1p121f))) {
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] = (float)(int8_t)((uint32_t)q[e / 4] >> (8 * (e % 4))) * s + (s - s);
        return;
    }
    const float off = s * -128.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const uint32_t w = (uint32_t)q[e / 4] ^ 0x80808080u;
        v[e] = __builtin_fmaf((float)((w >> (8 * (e % 4))) & 0xFFu), s, off);
    }
}

// dz of one row's eight outputs, the gate's (and, with a gate, the other half's in
// d[8 ..]).
template <int ACT, bool GATED>
__device__ __forceinline__ void dz8(const float dy[8], i32x2 cg, float sg, i32x2 cu, float su,
                                    float *d)
{
    float g[8], u[8];
    codes_times(cg, sg, g);
    if constexpr (GATED)
        codes_times(cu, su, u);
#pragma unroll
    for (int e = 0; e < 8; e++) {
        float value, slope;
        act_slope<ACT>(g[e], value, slope);
        if constexpr (GATED) {
            d[e] = dy[e] * u[e] * slope;
            d[8 + e] = dy[e] * value;
        } else {
            d[e] = dy[e] * slope;
        }
    }
}

template <int ACT, bool GATED, bool DY_BF16, bool DZ_BF16>
__global__ __launch_bounds__(256) void act_bwd_kernel(Args p)
{
    constexpr int H = GATED ? 2 : 1, E = 8 * H;
    __shared__ float red[2][kWaves - 1][E][kWave];
    const int lane = __lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int64_t F = p.a.F, N = p.N, M = p.a.M;
    const int64_t win = blockIdx.x;
    const int c0 = lane * 8;
    const int64_t left = F - win * kCols;
    const bool ok = c0 < left;          // then all eight are (F is a multiple of 16)
    // Lanes past the last output read it again; what they compute goes nowhere.
    const uint32_t c = ok ? c0 : (uint32_t)left - 8;
    float w[E], mx[E], sm[E];
#pragma unroll
    for (int e = 0; e < E; e++) {
        w[e] = p.a.sw ? p.a.sw[win * kCols + c + (e >= 8 ? F : 0) + e % 8] : 0.0f;
        if (!ok)
            w[e] = 0.0f;
        mx[e] = sm[e] = 0.0f;
    }
    struct Rows {
        Raw8<DY_BF16> dy[kBatch];
        i32x2 q[kBatch][H];
        float s[kBatch][H], px[kBatch];
    };
    // Rows past the last read it again, with a dy of zeros.
    auto load = [&](Rows &x, int64_t rb) {
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            const int64_t r = rb + u < M ? rb + u : M - 1;
            x.dy[u] = load_raw8<DY_BF16>(static_cast<const char *>(p.a.dy) + (r * F + win * kCols) * (DY_BF16 ? 2 : 4), c);
#pragma unroll
            for (int h = 0; h < H; h++) {
                x.q[u][h] = __builtin_nontemporal_load(
                    reinterpret_cast<const i32x2 *>(p.a.ck + r * N + h * F + win * kCols + c));
                x.s[u][h] = (p.a.ck_s + r * p.all + h * p.per + win * (kCols / kCkBlock))[c / kCkBlock];
            }
            x.px[u] = p.a.sx ? p.a.sx[r] : 0.0f;
        }
    };
    auto reduce = [&](const Rows &x, int64_t rb) {
        float d[kBatch][E], rm[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; u++) {
            float v[8];
            unpack8<DY_BF16>(x.dy[u], v);
#pragma unroll
            for (int e = 0; e < 8; e++)
                v[e] = rb + u < M ? v[e] : 0.0f;
            dz8<ACT, GATED>(v, x.q[u][0], x.s[u][0], x.q[u][H - 1], x.s[u][H - 1], d[u]);
            rm[u] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; e++)
                rm[u] = max_nan(rm[u], __builtin_fabsf(d[u][e] * w[e]));
            if (ok && rb + u < M) {
#pragma unroll
                for (int h = 0; h < H; h++) {
                    const int64_t at = (rb + u) * N + h * F + win * kCols;
                    if constexpr (DZ_BF16)
                        __builtin_nontemporal_store(
                            pack_bf16x8(d[u] + 8 * h),
                            reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(p.a.dz) + at + c));
                    else
                        store8(static_cast<float *>(p.a.dz) + at, c, d[u] + 8 * h);
                }
            }
        }
        // (Two rows' maxima at a time: the instruction takes three operands.)
#pragma unroll
        for (int e = 0; e < E; e++)
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                sm[e] = sm[e] + d[u][e];
                mx[e] = max_nan(mx[e], __builtin_fabsf(d[u][e] * x.px[u]));
            }
        if (p.a.sw) {
            float m = 0.0f;
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const float t = wave_all(rm[u], [](float a, float b) { return max_nan(a, b); });
                m = lane == u ? t : m;
            }
            if (lane < kBatch && rb + lane < M)
                p.rowpart[win * M + rb + lane] = m;
        }
    };
    // The next rows' loads are in flight while a batch is reduced.
    const int64_t step = (int64_t)gridDim.y * kWaves * kBatch;
    int64_t rb = ((int64_t)blockIdx.y * kWaves + wave) * kBatch;
    if (rb < M) {
        Rows one, two;
        load(one, rb);
        while (true) {
            load(two, rb + step);
            reduce(one, rb);
            if (rb + step >= M)
                break;
            load(one, rb + 2 * step);
            reduce(two, rb + step);
            rb += 2 * step;
            if (rb >= M)
                break;
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int e = 0; e < E; e++) {
            red[0][wave - 1][e][lane] = mx[e];
            red[1][wave - 1][e][lane] = sm[e];
        }
    }
    __syncthreads();
    if (wave > 0 || !ok)
        return;
#pragma unroll
    for (int k = 0; k < kWaves - 1; k++)
#pragma unroll
        for (int e = 0; e < E; e++) {
            mx[e] = max_nan(mx[e], red[0][k][e][lane]);
            sm[e] = sm[e] + red[1][k][e][lane];
        }
    float *out = p.colpart + 2 * (int64_t)blockIdx.y * N + win * kCols;
#pragma unroll
    for (int h = 0; h < H; h++) {
        store8(out + h * F, c, mx + 8 * h);
        store8(out + N + h * F, c, sm + 8 * h);
    }
}

// Partials -> s1, s2 and db.  A workgroup owns 64 columns, or, past the first
// ceil(N / 64) workgroups, 64 of the launch's rows: its 16 waves take every 16th row group (window) and
// are combined through LDS in a fixed order.
__global__ __launch_bounds__(1024) void act_bwd_scales_kernel(const float *__restrict__ rowpart, int wins,
                                                              const float *__restrict__ colpart, int groups,
                                                              int64_t M, int64_t nrows, int64_t N,
                                                              float *__restrict__ s1,
                                                              float *__restrict__ s2, float *__restrict__ db)
{
    __shared__ float red_max[16][64], red_sum[16][64];
    const int64_t cblocks = (N + 63) / 64;
    const bool rows = (int64_t)blockIdx.x >= cblocks;
    const int lc = threadIdx.x % 64, sl = threadIdx.x / 64;
    const int64_t c = ((int64_t)blockIdx.x - (rows ? cblocks : 0)) * 64 + lc;
    float m = 0.0f, sum = 0.0f;
    if (rows) {
        if (c < nrows) {
#pragma unroll 4
            for (int k = sl; k < wins; k += 16)
                m = max_nan(m, rowpart[k * M + c]);
        }
    } else if (c < N) {
#pragma unroll 4
        for (int g = sl; g < groups; g += 16) {
            m = max_nan(m, colpart[(2 * (int64_t)g) * N + c]);
            sum = sum + colpart[(2 * (int64_t)g + 1) * N + c];
        }
    }
    red_max[sl][lc] = m;
    red_sum[sl][lc] = sum;
    __syncthreads();
    if (sl != 0 || c >= (rows ? nrows : N))
        return;
#pragma unroll
    for (int i = 1; i < 16; i++) {
        m = max_nan(m, red_max[i][lc]);
        sum = sum + red_sum[i][lc];
    }
    if (rows) {
        s1[c] = m / 127.0f;
    } else {
        if (s2)
            s2[c] = m / 127.0f;
        if (db)
            db[c] = sum;
    }
}

// Windows of a row and row groups: about kGroups workgroups, of at least 32 rows (the
// partials of a group are 8 bytes per column, written and read), or if that leaves
// fewer than two workgroups per compute unit, of at least one batch per wave.
struct Shape {
    int64_t wins, groups;
};
Shape shape_of(int64_t M, int64_t F)
{
    const int64_t wins = (F + kCols - 1) / kCols, most = (M + kWaves * kBatch - 1) / (kWaves * kBatch);
    const int64_t few = (512 + wins - 1) / wins, all = (kGroups + wins - 1) / wins;
    int64_t groups = M / 32 > few ? M / 32 : few;
    groups = groups < all ? groups : all;
    return {wins, groups < most ? groups : most};
}

} // namespace

size_t act_bwd_bytes(int64_t M, int64_t F, bool gated)
{
    const Shape s = shape_of(M, F);
    const int64_t rows = (s.wins * M + 3) / 4 * 4;      // (16-byte steps)
    return (size_t)(rows + 2 * s.groups * F * (gated ? 2 : 1)) * 4;
}

void launch_act_bwd(const ActBackward &a, void *ws, hipStream_t st)
{
    const Shape sh = shape_of(a.M, a.F);
    Args p{};
    p.a = a;
    p.N = a.gated ? 2 * a.F : a.F;
    p.per = (a.F + kCkBlock - 1) / kCkBlock;
    p.all = a.gated ? 2 * p.per : p.per;
    p.rowpart = static_cast<float *>(ws);
    p.colpart = p.rowpart + (sh.wins * a.M + 3) / 4 * 4;
    auto go = [&](auto act, auto gated, auto dy, auto dz) {
        hipLaunchKernelGGL((act_bwd_kernel<decltype(act)::value, decltype(gated)::value, decltype(dy)::value,
                                           decltype(dz)::value>),
                           dim3((unsigned)sh.wins, (unsigned)sh.groups), dim3(kWaves * kWave), 0, st, p);
    };
    auto with_dz = [&](auto act, auto gated, auto dy) {
        a.dz_bf16 ? go(act, gated, dy, std::true_type()) : go(act, gated, dy, std::false_type());
    };
    auto with_dy = [&](auto act, auto gated) {
        a.dy_bf16 ? with_dz(act, gated, std::true_type()) : with_dz(act, gated, std::false_type());
    };
    auto with_act = [&](auto act) {
        a.gated ? with_dy(act, std::true_type()) : with_dy(act, std::false_type());
    };
    if (a.M > 0) {
        switch (a.act) {
        case QLIN_ACT_NONE: with_act(std::integral_constant<int, QLIN_ACT_NONE>()); break;
        case QLIN_ACT_RELU: with_act(std::integral_constant<int, QLIN_ACT_RELU>()); break;
        case QLIN_ACT_SILU: with_act(std::integral_constant<int, QLIN_ACT_SILU>()); break;
        case QLIN_ACT_GELU: with_act(std::integral_constant<int, QLIN_ACT_GELU>()); break;
        default: with_act(std::integral_constant<int, QLIN_ACT_GELU_TANH>()); break;
        }
    }
    // (s1 and its workgroups only where it is asked for.  A launch holds fewer than 2^32
    // threads: more rows than 2^27 take another, without columns.)
    if (!a.s1 && !a.s2 && !a.db)
        return;
    constexpr int64_t kRows = (int64_t)1 << 27;
    int64_t row = 0;
    do {
        const int64_t left = a.s1 ? a.M - row : 0, n = left < kRows ? left : kRows, cols = row ? 0 : p.N;
        hipLaunchKernelGGL(act_bwd_scales_kernel, dim3((unsigned)((cols + 63) / 64 + (n + 63) / 64)), dim3(1024), 0,
                           st, p.rowpart + row, (int)sh.wins, p.colpart, (int)sh.groups, a.M, n, cols,
                           a.s1 ? a.s1 + row : nullptr, a.s2, a.db);
        row += kRows;
    } while (a.s1 && row < a.M);
}

} // namespace qlin
