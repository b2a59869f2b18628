// Argument checks shared by the C-ABI entry points (host code).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "qlin.h"
#include "launch.hpp"

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
inline bool dtype_ok(int dt) { return dt == QLIN_F32 || dt == QLIN_BF16; }
inline bool dim16(int64_t v) { return v >= 16 && v % 16 == 0; }
inline bool hadamard_block_ok(int64_t cols, int b)
{
    return b >= 2 && b <= QLIN_MAX_HAD_BLOCK && pow2(b) && cols % b == 0;
}

// Optional pointers: 16-byte aligned when present.
inline bool opt_aligned(const void *p) { return p == nullptr || aligned16(p); }

// An array argument: non-null and 16-byte aligned unless it holds no element.
inline bool array_ok(const void *p, bool nonempty) { return nonempty ? (p && aligned16(p)) : opt_aligned(p); }

// a * b (and a * b * c) for non-negative sizes, saturated at INT64_MAX: a
// size check on the result then rejects the arguments as it would the exact
// product, and no argument can make the arithmetic overflow.
inline int64_t sat_mul(int64_t a, int64_t b)
{
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}
inline int64_t sat_mul(int64_t a, int64_t b, int64_t c) { return sat_mul(sat_mul(a, b), c); }

// Whether byte ranges [a, a + na) and [b, b + nb) intersect (empty ranges and
// null pointers never do).  Compared as integer addresses, ends saturated at
// the top of the address space.
inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    if (!a || !b || na <= 0 || nb <= 0)
        return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const uintptr_t xe = (uint64_t)na > UINTPTR_MAX - x ? UINTPTR_MAX : x + (uintptr_t)na;
    const uintptr_t ye = (uint64_t)nb > UINTPTR_MAX - y ? UINTPTR_MAX : y + (uintptr_t)nb;
    return x < ye && y < xe;
}

// Largest token count a call accepts (grid dimensions and int32 tile indices).
constexpr int64_t kMaxRows = (int64_t)1 << 30;

inline int finish()
{
    return hipGetLastError() == hipSuccess ? QLIN_OK : QLIN_EDEVICE;
}

// fl32(1 / sqrt(b)), the rotation's normalisation.
inline float hadamard_scale(int b) { return (float)(1.0 / sqrt((double)b)); }

inline hipStream_t as_stream(void *s) { return reinterpret_cast<hipStream_t>(s); }

// Shared checks of the three products: shapes, pointers, then the contraction
// bound.  'a_rows' / 'b_rows' tell whether the operands hold any element and
// 'out_rows' whether the output does.
inline int check_product(int op, const void *a, const void *b, void *out, int64_t M, int64_t N,
                         int64_t K, int64_t max_contraction = QLIN_MAX_CONTRACTION)
{
    if (M < 0 || !dim16(N) || !dim16(K))
        return QLIN_EINVAL;
    const bool has_m = M > 0;
    // forward and dX outputs have M rows; the dW output [N, K] exists for any M.
    const bool out_nonempty = op == QLIN_OP_DW ? true : has_m;
    const bool b_nonempty = op == QLIN_OP_DW ? has_m : true;
    if (!array_ok(a, has_m) || !array_ok(b, b_nonempty && has_m) || !array_ok(out, out_nonempty))
        return QLIN_EINVAL;
    const int64_t contraction = op == QLIN_OP_FWD ? K : (op == QLIN_OP_DX ? N : M);
    if (contraction > max_contraction || M > kMaxRows || N > kMaxRows || K > kMaxRows)
        return QLIN_EUNSUPPORTED;
    // The output's 256 x 256 tiles are counted (and indexed) as int.
    const int64_t rows = op == QLIN_OP_DW ? N : M, cols = op == QLIN_OP_FWD ? N : K;
    if (((rows + 255) / 256) * ((cols + 255) / 256) >= ((int64_t)1 << 31))
        return QLIN_EUNSUPPORTED;
    if (!qlin::product_addressable(op, M, N, K))
        return QLIN_EUNSUPPORTED;
    return QLIN_OK;
}

} // namespace
