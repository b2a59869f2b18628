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
#include <type_traits>

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

// Sixteen consecutive elements, as they lie in memory: the unit of this
// kernel's loads.
template <int X> struct Raw16 {
    static constexpr int kWords = X == X_I8 ? 1 : X == X_BF16 ? 2 : 4;
    i32x4 w[kWords];
};

template <int X> __device__ __forceinline__ Raw16<X> load16(const void *p, int64_t idx, bool ok)
{
    constexpr int kSize = X == X_I8 ? 1 : X == X_BF16 ? 2 : 4;
    Raw16<X> r;
#pragma unroll
    for (int q = 0; q < Raw16<X>::kWords; q++) {
        r.w[q] = i32x4{0, 0, 0, 0};
        if (ok)
            r.w[q] = *reinterpret_cast<const i32x4 *>(static_cast<const char *>(p) + idx * kSize + 16 * q);
    }
    return r;
}

// Elements 8 h .. 8 h + 7 of the sixteen as an MFMA operand.
template <int X, int H> __device__ __forceinline__ Frag<terms_of(X)> frag_of(const Raw16<X> &r)
{
    Frag<terms_of(X)> f;
    if constexpr (X == X_BF16) {
        f.t[0] = __builtin_bit_cast(bf16x8, r.w[H]);
    } else if constexpr (X == X_I8) {
        float v[8];
        codes_to_float(i32x2{r.w[0][2 * H], r.w[0][2 * H + 1]}, v);
        f.t[0] = round8(v);
    } else {
        float v[8];
        unpack8<false>({__builtin_bit_cast(f32x4, r.w[2 * H]), __builtin_bit_cast(f32x4, r.w[2 * H + 1])},
                       v);
        f = split8(v);
    }
    return f;
}

template <int X> __device__ __forceinline__ void floats_of(const Raw16<X> &r, float v[16])
{
    if constexpr (X == X_I8) {
        codes_to_float(i32x2{r.w[0][0], r.w[0][1]}, v);
        codes_to_float(i32x2{r.w[0][2], r.w[0][3]}, v + 8);
    } else if constexpr (X == X_BF16) {
        unpack8<true>({r.w[0]}, v);
        unpack8<true>({r.w[1]}, v + 8);
    } else {
#pragma unroll
        for (int e = 0; e < 16; e++)
            v[e] = __builtin_bit_cast(f32x4, r.w[e / 4])[e % 4];
    }
}

// out[m, r] = scale xs[m] sum_c x[m, c] w[id, r, c] for TB blocks of 16 tokens
// and RB of 16 ranks per workgroup; its waves take turns along the contraction
// and add their sums in LDS.  What bounds it is the read of x, so the loads
// are wide: of a chunk of 128 contraction indexes each of the four lane groups
// takes 32 in a row, a full line per row of INT8 codes, and multiplies them in
// four steps.  (The order inside a chunk is the same for x and w, which is all
// the product needs.)
template <int X, int W, int TB, int RB, int WAVES>
__global__ __launch_bounds__(WAVES *kWave) void adapter_shrink_kernel(ShrinkArgs a)
{
    __shared__ f32x4 red[WAVES * kWave];
    const int lane = __lane_id(), w = threadIdx.x / kWave;
    const int rb0 = blockIdx.y * RB * 16;
    int64_t m[TB], row[TB];
    int id[TB];
#pragma unroll
    for (int t = 0; t < TB; t++) {
        m[t] = ((int64_t)blockIdx.x * TB + t) * 16 + lane % 16;
        row[t] = (m[t] < a.M ? m[t] : a.M - 1) * a.C;
        id[t] = id_of(a.ids, m[t], a.M, a.L);
    }
    f32x4 acc[TB][RB];
#pragma unroll
    for (int t = 0; t < TB; t++)
#pragma unroll
        for (int b = 0; b < RB; b++)
            acc[t][b] = f32x4{0, 0, 0, 0};
    int left[TB];
#pragma unroll
    for (int t = 0; t < TB; t++)
        left[t] = id[t];
    while (true) {
        int cur = -1;
#pragma unroll
        for (int t = 0; t < TB; t++) {
            const uint64_t any = __ballot(left[t] >= 0);
            if (any)
                cur = __builtin_amdgcn_readlane(left[t], (int)__builtin_ctzll(any));
        }
        if (cur < 0)
            break;
        const int64_t wrow = ((int64_t)cur * a.R + rb0 + lane % 16) * a.C;
        f32x4 s[TB][RB];
#pragma unroll
        for (int t = 0; t < TB; t++)
#pragma unroll
            for (int b = 0; b < RB; b++)
                s[t][b] = f32x4{0, 0, 0, 0};
        for (int64_t k0 = (int64_t)w * 128; k0 < a.C; k0 += WAVES * 128) {
            const int64_t k = k0 + 32 * (lane / 16);
            Raw16<X> xr[TB][2];
            Raw16<W> wr[RB][2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const bool ok = k + 16 * h < a.C;
#pragma unroll
                for (int t = 0; t < TB; t++)
                    xr[t][h] = load16<X>(a.x, row[t] + k + 16 * h, ok);
#pragma unroll
                for (int b = 0; b < RB; b++)
                    wr[b][h] = load16<W>(a.w, wrow + (int64_t)16 * b * a.C + k + 16 * h,
                                         ok && rb0 + 16 * b + lane % 16 < a.R);
            }
            auto step = [&](auto H) {
                constexpr int h = decltype(H)::value;
                Frag<terms_of(X)> xf[TB];
#pragma unroll
                for (int t = 0; t < TB; t++)
                    xf[t] = frag_of<X, h % 2>(xr[t][h / 2]);
#pragma unroll
                for (int b = 0; b < RB; b++) {
                    const auto wf = frag_of<W, h % 2>(wr[b][h / 2]);
#pragma unroll
                    for (int t = 0; t < TB; t++)
                        s[t][b] = mfma(wf, xf[t], s[t][b]);
                }
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
        }
#pragma unroll
        for (int t = 0; t < TB; t++) {
            const bool mine = id[t] == cur;
            left[t] = mine ? -1 : left[t];
#pragma unroll
            for (int b = 0; b < RB; b++)
                acc[t][b] = mine ? s[t][b] : acc[t][b];
        }
    }
#pragma unroll
    for (int t = 0; t < TB; t++) {
        const float f = id[t] >= 0 ? a.scale[id[t]] * (a.xs ? a.xs[m[t]] : 1.0f) : 0.0f;
#pragma unroll
        for (int b = 0; b < RB; b++) {
            if (t + b > 0)
                __syncthreads();
            red[threadIdx.x] = acc[t][b];
            __syncthreads();
            const int r = rb0 + 16 * b + 4 * (lane / 16);
            if (w == (t * RB + b) % WAVES && m[t] < a.M && r < a.R) {
                f32x4 s = red[lane];
                for (int i = 1; i < WAVES; i++)
                    s += red[i * kWave + lane];
                *reinterpret_cast<f32x4 *>(a.out + m[t] * a.R + r) =
                    id[t] >= 0 ? s * f : f32x4{0, 0, 0, 0};
            }
        }
    }
}

// The same for a few tokens: one wave per token and rank, whose read of w (the
// ranks of one token's adapter in as many waves) is what takes the time.
template <int X, int W>
__global__ __launch_bounds__(256) void adapter_shrink_few_kernel(ShrinkArgs a)
{
    const int lane = __lane_id();
    const int64_t at = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
    const int64_t m = at / a.R;
    const int r = (int)(at % a.R);      // (R is a multiple of 4: one token per workgroup)
    const int id = id_of(a.ids, m, a.M, a.L);
    float s = 0.0f;
    if (id >= 0) {
        const int64_t x0 = m * a.C, w0 = ((int64_t)id * a.R + r) * a.C;
#pragma unroll 4
        for (int64_t k = lane * 16; k < a.C; k += kWave * 16) {
            const auto xr = load16<X>(a.x, x0 + k, true);
            const auto wr = load16<W>(a.w, w0 + k, true);
            float x[16], w[16];
            floats_of(xr, x);
            floats_of(wr, w);
#pragma unroll
            for (int e = 0; e < 16; e++)
                s = __builtin_fmaf(x[e], w[e], s);
        }
    }
    s = wave_all(s, [](float p, float q) { return p + q; });
    if (lane == 0)
        a.out[m * a.R + r] = id >= 0 ? s * (a.scale[id] * (a.xs ? a.xs[m] : 1.0f)) : 0.0f;
}

// Most tokens of the kernel above: it reads an adapter once per token.
constexpr int64_t kFewTokens = 32;

template <int X, int W, int TB, int RB, int WAVES> void go_shrink(const ShrinkArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.M + 16 * TB - 1) / (16 * TB)), (unsigned)((a.R + 16 * RB - 1) / (16 * RB)));
    hipLaunchKernelGGL((adapter_shrink_kernel<X, W, TB, RB, WAVES>), grid, dim3(WAVES * kWave), 0, st, a);
}

template <int X, bool WB> void run_shrink(const ShrinkArgs &a, hipStream_t st)
{
    constexpr int W = WB ? X_BF16 : X_F32;
    if (X == X_I8 && a.M <= kFewTokens) {
        hipLaunchKernelGGL((adapter_shrink_few_kernel<X_I8, W>), dim3((unsigned)(a.M * a.R / 4)), dim3(256),
                           0, st, a);
        return;
    }
    // Two token blocks share an adapter's operands; when that leaves compute
    // units without a workgroup, one block, ranks in workgroups of their own
    // and more waves along the contraction.
    const int64_t blocks = (a.M + 15) / 16;
    if (blocks >= 512)
        return a.R <= 16 ? go_shrink<X, W, 2, 1, 4>(a, st) : go_shrink<X, W, 2, 2, 4>(a, st);
    return a.R <= 16 || blocks < 128 ? go_shrink<X, W, 1, 1, 16>(a, st) : go_shrink<X, W, 1, 2, 8>(a, st);
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

struct PrepArgs {
    const void *a, *b;      // [L, R, K], [L, N, R]
    void *at, *bt;          // [L, K, R], [L, R, N]
    int64_t N, K, M;
    int L, R, slabs;
    const int32_t *start;
    Slab *table;            // [slabs]
    int32_t *first;         // [L + 1]: the first slab of each adapter
};

// dst [cols, rows] = src [rows, cols], one 32 x 32 tile.
template <typename T>
__device__ __forceinline__ void transpose_tile(const T *src, T *dst, int64_t rows, int64_t cols, int64_t r0,
                                               int64_t c0)
{
    __shared__ T tile[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
#pragma unroll
    for (int i = y; i < 32; i += 8)
        if (r0 + i < rows && c0 + x < cols)
            tile[i][x] = src[(r0 + i) * cols + c0 + x];
    __syncthreads();
#pragma unroll
    for (int i = y; i < 32; i += 8)
        if (c0 + i < cols && r0 + x < rows)
            dst[(c0 + i) * rows + r0 + x] = tile[x][i];
}

// What the backward kernels need first, in one launch: B transposed for the
// product with dY and A for dX's epilogue (both then have the contraction
// index contiguous), and the table of slabs.  Workgroup 0 of adapter 0 makes
// the table, 256 adapters at a time.
template <typename T> __global__ __launch_bounds__(256) void adapter_prep_kernel(PrepArgs p)
{
    const int t = threadIdx.x;
    if (blockIdx.x > 0) {
        const int64_t rt = (p.R + 31) / 32, nt = (p.N + 31) / 32, l = blockIdx.y;
        const int64_t k = blockIdx.x - 1;
        const int64_t sb = l * p.N * p.R, sa = l * p.K * p.R;
        if (k < rt * nt)
            transpose_tile(static_cast<const T *>(p.b) + sb, static_cast<T *>(p.bt) + sb, p.N, p.R,
                           k / rt * 32, k % rt * 32);
        else
            transpose_tile(static_cast<const T *>(p.a) + sa, static_cast<T *>(p.at) + sa, p.R, p.K,
                           (k - rt * nt) % rt * 32, (k - rt * nt) / rt * 32);
        return;
    }
    if (blockIdx.y > 0)
        return;
    __shared__ int sum[4];
    const int w = t / kWave, lane = __lane_id();
    for (int i = t; i < p.slabs; i += 256)
        p.table[i] = Slab{0, 0, 0, 0};
    int base = 0;
    for (int l0 = 0; l0 <= p.L; l0 += 256) {
        __syncthreads();        // the zeros above, and the last round's sums
        const int l = l0 + t;
        int64_t s0 = 0, s1 = 0;
        if (l < p.L) {
            s0 = p.start[l];
            s1 = p.start[l + 1];
            s0 = s0 < 0 ? 0 : s0 > p.M ? p.M : s0;
            s1 = s1 < s0 ? s0 : s1 > p.M ? p.M : s1;
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
        int before = base + s - n;
        for (int i = 0; i < 4; i++) {
            before += i < w ? sum[i] : 0;
            base += sum[i];
        }
        if (l <= p.L)
            p.first[l] = before < p.slabs ? before : p.slabs;
        for (int i = 0; i < n && before + i < p.slabs; i++) {
            const int64_t f = s0 + (int64_t)i * kSlab;
            p.table[before + i] = Slab{l, (int32_t)f, (int32_t)(s1 - f < kSlab ? s1 - f : kSlab), 0};
        }
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

// An LDS tile of 32 tokens by COLS bf16 values, rows as in memory.  The
// operands have the token index as the contraction, which the transposing read
// brings into a lane: in each 16-lane group lane s points at row s / 4, columns
// 4 (s % 4) of its block, and lane i gets the four rows of column i.  Rows are
// 32 bytes apart in the banks and every eight of them another 128, so the 64
// lanes of a read fall on all banks twice.
template <int COLS> struct TokenTile {
    static constexpr int kRow = COLS + 16;
    static constexpr int kSize = 32 * kRow + 3 * 64;
    __device__ static __forceinline__ int at(int row, int col) { return row * kRow + (row / 8) * 64 + col; }

    // Columns c0 .. c0 + 15, all 32 tokens, as an MFMA operand.
    __device__ static __forceinline__ bf16x8 operand(const uint16_t *tile, int c0)
    {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int s = __lane_id() % 16, g = __lane_id() / 16;
        s16x4 h[2];
#pragma unroll
        for (int k = 0; k < 2; k++)
            h[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(tile + at(8 * g + 4 * k + s / 4, c0 + 4 * (s % 4))));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// part[slab] = sum over the slab's tokens of p^T x, for 256 columns: 64 per
// wave.  32 tokens at a time are brought into LDS, split into bf16 terms on
// the way; the next ones' loads are in flight meanwhile.  The read of x bounds
// it.
template <int X, bool TRANS, int RB>
__global__ __launch_bounds__(256) void adapter_outer_kernel(OuterArgs a)
{
    constexpr int XT = terms_of(X);
    using XTile = TokenTile<256>;
    using PTile = TokenTile<RB * 16>;
    __shared__ __attribute__((aligned(16))) uint16_t xs[XT][XTile::kSize];
    __shared__ __attribute__((aligned(16))) uint16_t ps[3][PTile::kSize];
    const Slab s = a.table[blockIdx.y];
    if (s.rows <= 0)
        return;
    const int t = threadIdx.x, w = t / kWave, lane = __lane_id();
    const int64_t c0 = (int64_t)blockIdx.x * 256;
    f32x4 acc[4][RB];
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int r = 0; r < RB; r++)
            acc[b][r] = f32x4{0, 0, 0, 0};
    // Thread t brings 32 columns of token t / 8, and two ranks in 16 of p.
    const int row = t / 8, xc = (t % 8) * 32, pc = (t % 8) * 2;
    auto token = [&](int i0) {
        const int i = i0 + row;
        const int64_t m = i < s.rows ? a.order[s.first + i] : -1;
        return m >= 0 && m < a.M ? m : (int64_t)-1;
    };
    Raw16<X> xr[2];
    f32x2 pr[RB];
    float f = 0.0f;
    auto load = [&](int64_t m) {
        const bool live = m >= 0;
        const int64_t mm = live ? m : 0;
#pragma unroll
        for (int h = 0; h < 2; h++)
            xr[h] = load16<X>(a.x, mm * a.C + c0 + xc + 16 * h, live && c0 + xc + 16 * h < a.C);
#pragma unroll
        for (int r = 0; r < RB; r++) {
            pr[r] = f32x2{0, 0};
            if (live && 16 * r + pc < a.R)
                pr[r] = *reinterpret_cast<const f32x2 *>(a.p + mm * a.R + 16 * r + pc);
        }
        f = live && a.ps ? a.ps[mm] : 1.0f;
    };
    int64_t next = token(0);
    load(next);
    next = token(32);
    for (int i0 = 0; i0 < s.rows; i0 += 32) {
        __syncthreads();
        auto put = [&](auto H) {
            constexpr int h = decltype(H)::value;
            const auto fr = frag_of<X, h % 2>(xr[h / 2]);
#pragma unroll
            for (int q = 0; q < XT; q++)
                *reinterpret_cast<bf16x8 *>(&xs[q][XTile::at(row, xc + 8 * h)]) = fr.t[q];
        };
        put(std::integral_constant<int, 0>{});
        put(std::integral_constant<int, 1>{});
        put(std::integral_constant<int, 2>{});
        put(std::integral_constant<int, 3>{});
#pragma unroll
        for (int r = 0; r < RB; r++) {
            float v0 = pr[r][0] * f, v1 = pr[r][1] * f;
#pragma unroll
            for (int q = 0; q < 3; q++) {
                const uint32_t b = pack_bf16x2(v0, v1);
                *reinterpret_cast<uint32_t *>(&ps[q][PTile::at(row, 16 * r + pc)]) = b;
                v0 = v0 - bf16_lo(b);
                v1 = v1 - bf16_hi(b);
            }
        }
        __syncthreads();
        load(next);             // (zeros after the last tokens)
        next = token(i0 + 64);
        Frag<XT> xf[4];
#pragma unroll
        for (int b = 0; b < 4; b++)
#pragma unroll
            for (int q = 0; q < XT; q++)
                xf[b].t[q] = XTile::operand(xs[q], w * 64 + 16 * b);
#pragma unroll
        for (int r = 0; r < RB; r++) {
            Frag<3> pf;
#pragma unroll
            for (int q = 0; q < 3; q++)
                pf.t[q] = PTile::operand(ps[q], 16 * r);
#pragma unroll
            for (int b = 0; b < 4; b++)
                acc[b][r] = TRANS ? mfma(pf, xf[b], acc[b][r]) : mfma(xf[b], pf, acc[b][r]);
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * a.R * a.C;
#pragma unroll
    for (int b = 0; b < 4; b++)
#pragma unroll
        for (int rb = 0; rb < RB; rb++) {
            const int64_t cb = c0 + w * 64 + 16 * b;
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
    const dim3 grid((unsigned)((a.C + 255) / 256), (unsigned)slabs), block(256);
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
// Both gradients in one launch: the workgroups from the first sa / 1024 on are
// B's.
__global__ __launch_bounds__(256) void adapter_sum_kernel(const float *__restrict__ pa, int64_t sa,
                                                          float *__restrict__ da,
                                                          const float *__restrict__ pb, int64_t sb,
                                                          float *__restrict__ db,
                                                          const int32_t *__restrict__ first)
{
    const int64_t na = (sa + 1023) / 1024;
    const bool is_a = (int64_t)blockIdx.x < na;
    const float *part = is_a ? pa : pb;
    float *out = is_a ? da : db;
    const int64_t size = is_a ? sa : sb;
    const int64_t i = ((is_a ? blockIdx.x : blockIdx.x - na) * 256 + threadIdx.x) * 4;
    if (i >= size)
        return;
    const int64_t l = blockIdx.y;
    const int k0 = first[l], k1 = first[l + 1];
    f32x4 s = {0, 0, 0, 0};
#pragma unroll 4
    for (int k = k0; k < k1; k++)
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
    size_t bt, at, v, table, first, pa, pb, end;
};

static BwdLayout bwd_layout(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    const size_t slabs = (size_t)slabs_of(M, L);
    BwdLayout o;
    o.bt = 0;
    o.at = round256(o.bt + (size_t)L * R * N * 4);
    o.v = round256(o.at + (size_t)L * R * K * 4);
    o.table = round256(o.v + (size_t)M * R * 4);
    o.first = round256(o.table + slabs * sizeof(Slab));
    o.pa = round256(o.first + ((size_t)L + 1) * 4);
    o.pb = round256(o.pa + slabs * (size_t)R * K * 4);
    o.end = round256(o.pb + slabs * (size_t)R * N * 4);
    return o;
}

size_t adapter_bwd_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R)
{
    return bwd_layout(M, N, K, L, R).end;
}

AdapterEpilogue launch_adapter_bwd_v(const AdapterArgs &g, const void *dy, bool dy_bf16,
                                     const int32_t *start, void *ws, hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    const BwdLayout o = bwd_layout(g.M, g.N, g.K, g.L, g.R);
    const PrepArgs p{g.a, g.b, w + o.at, w + o.bt, g.N, g.K, g.M, g.L, g.R, (int)slabs_of(g.M, g.L), start,
                     reinterpret_cast<Slab *>(w + o.table), reinterpret_cast<int32_t *>(w + o.first)};
    const int64_t tiles = (int64_t)((g.R + 31) / 32) * ((g.N + 31) / 32 + (g.K + 31) / 32);
    const dim3 grid((unsigned)(g.M > 0 ? 1 + tiles : 1), (unsigned)g.L);
    if (g.bf16)
        hipLaunchKernelGGL(adapter_prep_kernel<uint16_t>, grid, dim3(256), 0, st, p);
    else
        hipLaunchKernelGGL(adapter_prep_kernel<uint32_t>, grid, dim3(256), 0, st, p);
    const ShrinkArgs s{dy,  nullptr, w + o.bt, g.scale, g.ids, g.M, g.N,
                       g.L, g.R,     reinterpret_cast<float *>(w + o.v)};
    if (g.M > 0) {
        if (dy_bf16)
            g.bf16 ? run_shrink<X_BF16, true>(s, st) : run_shrink<X_BF16, false>(s, st);
        else
            g.bf16 ? run_shrink<X_F32, true>(s, st) : run_shrink<X_F32, false>(s, st);
    }
    return AdapterEpilogue{s.out, w + o.at, g.ids, g.L, g.R, g.bf16};
}

void launch_adapter_bwd_w(const AdapterArgs &g, const void *dy, bool dy_bf16, const int8_t *qx,
                          const float *sx, const float *u, const int32_t *order, float *da, float *db,
                          void *ws, hipStream_t st)
{
    char *w = static_cast<char *>(ws);
    const BwdLayout o = bwd_layout(g.M, g.N, g.K, g.L, g.R);
    const int slabs = (int)slabs_of(g.M, g.L);
    const Slab *table = reinterpret_cast<const Slab *>(w + o.table);
    float *pa = reinterpret_cast<float *>(w + o.pa), *pb = reinterpret_cast<float *>(w + o.pb);
    const float *v = reinterpret_cast<const float *>(w + o.v);
    if (g.M > 0) {
        run_outer<X_I8, false>(OuterArgs{v, sx, qx, order, table, g.M, g.K, g.R, pa}, slabs, st);
        const OuterArgs b{u, nullptr, dy, order, table, g.M, g.N, g.R, pb};
        dy_bf16 ? run_outer<X_BF16, true>(b, slabs, st) : run_outer<X_F32, true>(b, slabs, st);
    }
    const int64_t sa = (int64_t)g.R * g.K, sb = (int64_t)g.R * g.N;
    hipLaunchKernelGGL(adapter_sum_kernel, dim3((unsigned)((sa + 1023) / 1024 + (sb + 1023) / 1024), (unsigned)g.L),
                       dim3(256), 0, st, pa, sa, da, pb, sb, db,
                       reinterpret_cast<const int32_t *>(w + o.first));
}

} // namespace qlin
