// Low-rank adapters of many requests beside one shared INT8 projection.
//
// Token m has the adapter l = ids[m] (none if that is outside [0, L)); its
// matrices A[l] [R, K] and B[l] [N, R] and a factor scale[l].  The adapters
// read the projection's own INT8 input, x^ = sx q, in the basis of the codes
// (rotated where the projection's weight is), so a layer keeps one copy of
// its input, of one byte per element, for the projection and the adapters.
//
//   u = scale (x^ A^T)      y  = sx sw acc + bias + u B^T
//   v = scale (dY B)        dx = rotate(sg acc + v A)
//   dA[l] = sum over l's tokens of v^T x^     dB[l] = the same of dY^T u
//
// The products run on v_mfma_f32_16x16x32_bf16 with fp32 sums.  INT8 codes
// are exact in bf16; an fp32 operand is split into three bf16 terms, which hold
// its 24 bits, and a product of two such operands keeps the six partial
// products above 2^-24.  (Two terms and three products were 2.5 to 5 times as
// far from the 64-bit result as fp32 products are.)  Every lane of an accumulator belongs to one token, so the rows of a
// 16-token block that have another adapter are dropped by a select and never
// meet its matrices' values (a NaN in one adapter stays with its tokens).
#include "adapter_frag.hpp"
#include "common.hpp"
#include "launch.hpp"
#include "lowp.hpp"

namespace qlin {

namespace {

// ------------------------------------------------------------------ shrink

struct ShrinkArgs {
    const void *x;          // [M, C]
    const float *xs;        // [M] row scales of INT8 codes, or null
    const void *w;          // [L, R, C]
    const float *scale;     // [L]
    const int32_t *ids;
    int64_t M, C;
    int L, R;
    float *out;             // [M, R]
};

// out[m, r] = scale xs[m] sum_c x[m, c] w[id, r, c].  A workgroup holds 16
// tokens; its waves take turns along the contraction and add their sums in
// LDS.
template <int X, bool WB, int RB>
__global__ __launch_bounds__(1024) void adapter_shrink_kernel(ShrinkArgs a)
{
    constexpr int W = WB ? X_BF16 : X_F32;
    extern __shared__ f32x4 red[];      // [waves][64]
    const int lane = __lane_id(), w = threadIdx.x / kWave, waves = blockDim.x / kWave;
    const int64_t m = (int64_t)blockIdx.x * 16 + lane % 16;
    const int64_t mc = m < a.M ? m : a.M - 1;
    const int id = id_of(a.ids, m, a.M, a.L);
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; b++)
        acc[b] = f32x4{0, 0, 0, 0};
    for_adapters(id, [&](int cur, bool mine) {
        f32x4 t[RB];
#pragma unroll
        for (int b = 0; b < RB; b++)
            t[b] = f32x4{0, 0, 0, 0};
        for (int64_t k0 = (int64_t)w * 32; k0 < a.C; k0 += (int64_t)waves * 32) {
            const int64_t k = k0 + 8 * (lane / 16);
            const bool ok = k < a.C;
            const auto xf = load_frag<X>(a.x, mc * a.C + k, ok);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                const int r = 16 * b + lane % 16;
                const auto wf = load_frag<W>(a.w, ((int64_t)cur * a.R + r) * a.C + k, ok && r < a.R);
                t[b] = mfma(wf, xf, t[b]);
            }
        }
#pragma unroll
        for (int b = 0; b < RB; b++)
            acc[b] = mine ? t[b] : acc[b];
    });
    const float f = id >= 0 ? a.scale[id] * (a.xs ? a.xs[m] : 1.0f) : 0.0f;
#pragma unroll
    for (int b = 0; b < RB; b++) {
        if (b > 0)
            __syncthreads();
        red[threadIdx.x] = acc[b];
        __syncthreads();
        const int r = 16 * b + 4 * (lane / 16);
        if (w == 0 && m < a.M && r < a.R) {
            f32x4 s = red[lane];
            for (int i = 1; i < waves; i++)
                s += red[i * kWave + lane];
            *reinterpret_cast<f32x4 *>(a.out + m * a.R + r) =
                id >= 0 ? s * f : f32x4{0, 0, 0, 0};
        }
    }
}

template <int X, bool WB> void run_shrink(const ShrinkArgs &a, hipStream_t st)
{
    const int64_t blocks = (a.M + 15) / 16;
    const int waves = blocks >= 512 ? 4 : 16;
    const dim3 grid((unsigned)blocks), block(waves * kWave);
    const size_t lds = (size_t)waves * kWave * sizeof(f32x4);
    if (a.R <= 16)
        hipLaunchKernelGGL((adapter_shrink_kernel<X, WB, 1>), grid, block, lds, st, a);
    else if (a.R <= 32)
        hipLaunchKernelGGL((adapter_shrink_kernel<X, WB, 2>), grid, block, lds, st, a);
    else if (a.R <= 64)
        hipLaunchKernelGGL((adapter_shrink_kernel<X, WB, 4>), grid, block, lds, st, a);
    else
        hipLaunchKernelGGL((adapter_shrink_kernel<X, WB, 8>), grid, block, lds, st, a);
}

// --------------------------------------------------------------- transpose

// dst [L, cols, rows] = src [L, rows, cols] transposed, 32 x 32 tiles.
template <typename T>
__global__ __launch_bounds__(256) void adapter_transpose_kernel(const T *__restrict__ src,
                                                                T *__restrict__ dst, int64_t rows,
                                                                int64_t cols)
{
    __shared__ T tile[32][33];
    const int64_t l = blockIdx.z * rows * cols;
    const int64_t r0 = (int64_t)blockIdx.y * 32, c0 = (int64_t)blockIdx.x * 32;
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
#pragma unroll
    for (int i = y; i < 32; i += 8)
        if (r0 + i < rows && c0 + x < cols)
            tile[i][x] = src[l + (r0 + i) * cols + c0 + x];
    __syncthreads();
#pragma unroll
    for (int i = y; i < 32; i += 8)
        if (c0 + i < cols && r0 + x < rows)
            dst[l + (c0 + i) * rows + r0 + x] = tile[x][i];
}

void run_transpose(const void *src, void *dst, bool bf, int64_t L, int64_t rows, int64_t cols,
                   hipStream_t st)
{
    const dim3 grid((unsigned)((cols + 31) / 32), (unsigned)((rows + 31) / 32), (unsigned)L);
    if (bf)
        hipLaunchKernelGGL(adapter_transpose_kernel<uint16_t>, grid, dim3(256), 0, st,
                           static_cast<const uint16_t *>(src), static_cast<uint16_t *>(dst), rows, cols);
    else
        hipLaunchKernelGGL(adapter_transpose_kernel<uint32_t>, grid, dim3(256), 0, st,
                           static_cast<const uint32_t *>(src), static_cast<uint32_t *>(dst), rows, cols);
}

// ------------------------------------------------------- grouping of tokens

// A stable counting sort of the tokens by adapter, in one workgroup: each of 8
// waves counts its own run of tokens, the counts become first places (adapter
// by adapter, and for one adapter wave by wave), and each wave places its
// tokens 64 at a time, one adapter among them after another.  Tokens without
// an adapter come last.
constexpr int kGroupWaves = 8;

__global__ __launch_bounds__(kGroupWaves *kWave) void adapter_group_kernel(const int32_t *__restrict__ ids,
                                                                           int64_t M, int L,
                                                                           int32_t *__restrict__ order,
                                                                           int32_t *__restrict__ start)
{
    __shared__ int count[kGroupWaves][kMaxAdapters + 1];
    __shared__ int total[kMaxAdapters + 2];
    const int bins = L + 1, t = threadIdx.x, w = t / kWave, lane = __lane_id();
    for (int i = t; i < kGroupWaves * bins; i += kGroupWaves * kWave)
        count[i / bins][i % bins] = 0;
    __syncthreads();
    const int64_t per = (M + kGroupWaves - 1) / kGroupWaves;
    const int64_t r0 = w * per < M ? w * per : M, r1 = r0 + per < M ? r0 + per : M;
    auto bin_of = [&](int64_t m) {
        const int id = ids[m];
        return id >= 0 && id < L ? id : L;
    };
    for (int64_t m = r0 + lane; m < r1; m += kWave)
        atomicAdd(&count[w][bin_of(m)], 1);
    __syncthreads();
    for (int b = t; b < bins; b += kGroupWaves * kWave) {
        int s = 0;
        for (int i = 0; i < kGroupWaves; i++)
            s += count[i][b];
        total[b] = s;
    }
    __syncthreads();
    if (w == 0) {       // exclusive prefix sums of the totals, 64 bins at a time
        int before = 0;
        for (int b0 = 0; b0 < bins; b0 += kWave) {
            const int v = b0 + lane < bins ? total[b0 + lane] : 0;
            int s = v;
            for (int o = 1; o < kWave; o <<= 1) {
                const int x = __shfl_up(s, o);
                s += lane >= o ? x : 0;
            }
            if (b0 + lane < bins)
                total[b0 + lane] = before + s - v;
            before += __shfl(s, kWave - 1);
        }
    }
    __syncthreads();
    for (int b = t; b < bins; b += kGroupWaves * kWave) {
        int s = total[b];
        start[b] = s;       // start[L]: the first token without an adapter
        for (int i = 0; i < kGroupWaves; i++) {
            const int c = count[i][b];
            count[i][b] = s;
            s += c;
        }
    }
    __syncthreads();
    for (int64_t m0 = r0; m0 < r1; m0 += kWave) {
        const int64_t m = m0 + lane;
        const int b = m < r1 ? bin_of(m) : -1;
        uint64_t left = __ballot(b >= 0);
        while (left) {
            const int cur = __builtin_amdgcn_readlane(b, (int)__builtin_ctzll(left));
            const uint64_t mask = __ballot(b == cur);
            const int first = count[w][cur];
            if (b == cur)
                order[first + __popcll(mask & ((1ull << lane) - 1))] = (int32_t)m;
            if (lane == 0)
                count[w][cur] = first + __popcll(mask);
            left &= ~mask;
        }
    }
}

// ------------------------------------------------------- adapter gradients

// The tokens of an adapter are split into slabs of kSlab; a table entry says
// which adapter a slab has and where its tokens lie in the grouped order.
constexpr int kSlab = 512;

struct Slab {
    int32_t adapter, first, rows, pad;
};

// table[slabs], then first[L + 1]: the first slab of each adapter.
__global__ __launch_bounds__(1024) void adapter_slab_kernel(const int32_t *__restrict__ start, int64_t M,
                                                            int L, int slabs, Slab *__restrict__ table,
                                                            int32_t *__restrict__ first)
{
    __shared__ int sum[16];
    const int t = threadIdx.x, w = t / kWave, lane = __lane_id();
    for (int i = t; i < slabs; i += 1024)
        table[i] = Slab{0, 0, 0, 0};
    // (kMaxAdapters < 1024: one adapter per thread.)
    int64_t s0 = 0, s1 = 0;
    if (t < L) {
        s0 = start[t];
        s1 = start[t + 1];
        s0 = s0 < 0 ? 0 : s0 > M ? M : s0;
        s1 = s1 < s0 ? s0 : s1 > M ? M : s1;
    }
    const int n = (int)((s1 - s0 + kSlab - 1) / kSlab);
    int s = n;
    for (int o = 1; o < kWave; o <<= 1) {
        const int x = __shfl_up(s, o);
        s += lane >= o ? x : 0;
    }
    if (lane == kWave - 1)
        sum[w] = s;
    __syncthreads();
    int before = s - n;
    for (int i = 0; i < w; i++)
        before += sum[i];
    if (t <= L)
        first[t] = before < slabs ? before : slabs;
    for (int i = 0; i < n && before + i < slabs; i++) {
        const int64_t f = s0 + (int64_t)i * kSlab;
        table[before + i] = Slab{t, (int32_t)f, (int32_t)(s1 - f < kSlab ? s1 - f : kSlab), 0};
    }
}

struct OuterArgs {
    const float *p;         // [M, R]
    const float *ps;        // [M] factors of p's rows, or null
    const void *x;          // [M, C]
    const int32_t *order;
    const Slab *table;
    int64_t M, C;
    int R;
    float *part;            // per slab: [R, C], or [C, R] (TRANS)
};

// part[slab] = sum over the slab's tokens of p^T x, for 128 columns.  Both
// operands are brought into LDS with the token index contiguous, 32 tokens at
// a time.
template <int X, bool TRANS, int RB>
__global__ __launch_bounds__(256) void adapter_outer_kernel(OuterArgs a)
{
    constexpr int XT = terms_of(X), kStride = 40;
    __shared__ __attribute__((aligned(16))) uint16_t xs[XT][128 * kStride];
    __shared__ __attribute__((aligned(16))) uint16_t ps[3][RB * 16 * kStride];
    const Slab s = a.table[blockIdx.y];
    if (s.rows <= 0)
        return;
    const int t = threadIdx.x, w = t / kWave, lane = __lane_id();
    const int64_t c0 = (int64_t)blockIdx.x * 128;
    f32x4 acc[2][RB] = {};
    const int row = t / 8, xc = (t % 8) * 16;
    for (int i0 = 0; i0 < s.rows; i0 += 32) {
        const int i = i0 + row;
        int64_t m = i < s.rows ? a.order[s.first + i] : -1;
        const bool live = m >= 0 && m < a.M;
        m = live ? m : 0;
        const float f = live && a.ps ? a.ps[m] : 1.0f;
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const bool ok = live && c0 + xc < a.C;
            const auto fr = load_frag<X>(a.x, m * a.C + c0 + xc + 8 * h, ok);
#pragma unroll
            for (int q = 0; q < XT; q++) {
                const u16x8 bits = __builtin_bit_cast(u16x8, fr.t[q]);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    xs[q][(xc + 8 * h + e) * kStride + row] = bits[e];
            }
        }
        for (int r = t % 8; r < RB * 16; r += 8) {
            float v = live && r < a.R ? a.p[m * a.R + r] * f : 0.0f;
#pragma unroll
            for (int q = 0; q < 3; q++) {
                const uint32_t t = pack_bf16x2(v, 0.0f);
                ps[q][r * kStride + row] = (uint16_t)t;
                v = v - bf16_lo(t);
            }
        }
        __syncthreads();
        Frag<XT> xf[2];
#pragma unroll
        for (int b = 0; b < 2; b++)
#pragma unroll
            for (int q = 0; q < XT; q++)
                xf[b].t[q] = *reinterpret_cast<const bf16x8 *>(
                    &xs[q][(w * 32 + 16 * b + lane % 16) * kStride + 8 * (lane / 16)]);
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            Frag<3> pf;
#pragma unroll
            for (int q = 0; q < 3; q++)
                pf.t[q] = *reinterpret_cast<const bf16x8 *>(
                    &ps[q][(16 * rb + lane % 16) * kStride + 8 * (lane / 16)]);
#pragma unroll
            for (int b = 0; b < 2; b++)
                acc[b][rb] = TRANS ? mfma(pf, xf[b], acc[b][rb]) : mfma(xf[b], pf, acc[b][rb]);
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * a.R * a.C;
#pragma unroll
    for (int b = 0; b < 2; b++)
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            const int64_t cb = c0 + w * 32 + 16 * b;
            if (TRANS) {
                const int64_t c = cb + lane % 16;
                const int r = 16 * rb + 4 * (lane / 16);
                if (c < a.C && r < a.R)
                    *reinterpret_cast<f32x4 *>(part + c * a.R + r) = acc[b][rb];
            } else {
                const int64_t c = cb + 4 * (lane / 16);
                const int r = 16 * rb + lane % 16;
                if (c < a.C && r < a.R)
                    *reinterpret_cast<f32x4 *>(part + r * a.C + c) = acc[b][rb];
            }
        }
}

template <int X, bool TRANS> void run_outer(const OuterArgs &a, int slabs, hipStream_t st)
{
    const dim3 grid((unsigned)((a.C + 127) / 128), (unsigned)slabs), block(256);
    if (a.R <= 16)
        hipLaunchKernelGGL((adapter_outer_kernel<X, TRANS, 1>), grid, block, 0, st, a);
    else if (a.R <= 32)
        hipLaunchKernelGGL((adapter_outer_kernel<X, TRANS, 2>), grid, block, 0, st, a);
    else if (a.R <= 64)
        hipLaunchKernelGGL((adapter_outer_kernel<X, TRANS, 4>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((adapter_outer_kernel<X, TRANS, 8>), grid, block, 0, st, a);
}

// out[l] = the sum of l's slabs, in order; zeros for an adapter without tokens.
__global__ __launch_bounds__(256) void adapter_sum_kernel(const float *__restrict__ part,
                                                          const int32_t *__restrict__ first, int64_t size,
                                                          float *__restrict__ out)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= size)
        return;
    const int64_t l = blockIdx.y;
    f32x4 s = {0, 0, 0, 0};
    for (int k = first[l]; k < first[l + 1]; k++)
        s += *reinterpret_cast<const f32x4 *>(part + k * size + i);
    *reinterpret_cast<f32x4 *>(out + l * size + i) = s;
}

} // namespace

void launch_adapter_u(const AdapterArgs &g, const int8_t *qx, const float *sx, float *u,
                      hipStream_t st)
{
    const ShrinkArgs s{qx, sx, g.a, g.scale, g.ids, g.M, g.K, g.L, g.R, u};
    g.bf16 ? run_shrink<X_I8, true>(s, st) : run_shrink<X_I8, false>(s, st);
}

void launch_adapter_group(const int32_t *ids, int64_t M, int L, int32_t *order, int32_t *start,
                          hipStream_t st)
{
    hipLaunchKernelGGL(adapter_group_kernel, dim3(1), dim3(kGroupWaves * kWave), 0, st, ids, M, L, order,
                       start);
}

static int64_t slabs_of(int64_t M, int64_t L) { return M / kSlab + (M < L ? M : L); }

static size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Offsets of a backward call's workspace.
struct BwdLayout {
    size_t bt, at, v, table, first, part, end;
};

static BwdLayout bwd_layout(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    const size_t slabs = (size_t)slabs_of(M, L), C = (size_t)(N > K ? N : K);
    BwdLayout o;
    o.bt = 0;
    o.at = round256(o.bt + (size_t)L * R * N * 4);
    o.v = round256(o.at + (size_t)L * R * K * 4);
    o.table = round256(o.v + (size_t)M * R * 4);
    o.first = round256(o.table + slabs * sizeof(Slab));
    o.part = round256(o.first + ((size_t)L + 1) * 4);
    o.end = round256(o.part + slabs * (size_t)R * C * 4);
    return o;
}

size_t adapter_bwd_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    return bwd_layout(M, N, K, L, R).end;
}

AdapterEpilogue launch_adapter_bwd_v(const AdapterArgs &g, const void *dy, bool dy_bf16, void *ws,
                                     hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    const BwdLayout o = bwd_layout(g.M, g.N, g.K, g.L, g.R);
    run_transpose(g.b, w + o.bt, g.bf16, g.L, g.N, g.R, st);
    run_transpose(g.a, w + o.at, g.bf16, g.L, g.R, g.K, st);
    const ShrinkArgs s{dy,  nullptr, w + o.bt, g.scale, g.ids, g.M, g.N,
                       g.L, g.R,     reinterpret_cast<float *>(w + o.v)};
    if (dy_bf16)
        g.bf16 ? run_shrink<X_BF16, true>(s, st) : run_shrink<X_BF16, false>(s, st);
    else
        g.bf16 ? run_shrink<X_F32, true>(s, st) : run_shrink<X_F32, false>(s, st);
    return AdapterEpilogue{s.out, w + o.at, g.ids, g.L, g.R, g.bf16};
}

void launch_adapter_bwd_w(const AdapterArgs &g, const void *dy, bool dy_bf16, const int8_t *qx,
                          const float *sx, const float *u, const int32_t *order, const int32_t *start,
                          float *da, float *db, void *ws, hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    const BwdLayout o = bwd_layout(g.M, g.N, g.K, g.L, g.R);
    const int slabs = (int)slabs_of(g.M, g.L);
    Slab *table = reinterpret_cast<Slab *>(w + o.table);
    int32_t *first = reinterpret_cast<int32_t *>(w + o.first);
    float *part = reinterpret_cast<float *>(w + o.part);
    const float *v = reinterpret_cast<const float *>(w + o.v);
    hipLaunchKernelGGL(adapter_slab_kernel, dim3(1), dim3(1024), 0, st, start, g.M, g.L, slabs, table,
                       first);
    auto sum = [&](int64_t size, float *out) {
        hipLaunchKernelGGL(adapter_sum_kernel, dim3((unsigned)((size / 4 + 255) / 256), (unsigned)g.L),
                           dim3(256), 0, st, part, first, size, out);
    };
    if (g.M > 0)
        run_outer<X_I8, false>(OuterArgs{v, sx, qx, order, table, g.M, g.K, g.R, part}, slabs, st);
    sum((int64_t)g.R * g.K, da);
    const OuterArgs b{u, nullptr, dy, order, table, g.M, g.N, g.R, part};
    if (g.M > 0)
        dy_bf16 ? run_outer<X_BF16, true>(b, slabs, st) : run_outer<X_F32, true>(b, slabs, st);
    sum((int64_t)g.R * g.N, db);
}

} // namespace qlin
