// Argument checks shared by the host files of the operators: each returns a status with
// its message recorded (nothing is enqueued, no pointer followed).
#pragma once
#include <stdint.h>

#include <numeric>

#include "../../include/moe_ops.h"
#include "ops.h"
#include "status.h"

namespace moe {
namespace checks {

inline bool misaligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Device memory that a call reads or writes: `rows` pieces of `width` bytes, `stride`
// bytes apart (nothing when p is NULL or a count is 0).
struct Range {
    const char* what;
    const void* p;
    uint64_t rows, width, stride;
    bool written;
};

inline Range dense(const char* what, const void* p, uint64_t bytes, bool written) {
    return Range{what, p, 1, bytes, 0, written};
}

// rows x width elements with a row stride (of one row, the stride is not looked at).
inline Range strided(const char* what, const void* p, int64_t rows, int64_t width, int64_t stride, int elem, bool written) {
    return Range{what, p, (uint64_t)rows, (uint64_t)(width * elem), rows > 1 ? (uint64_t)(stride * elem) : 0, written};
}

// Whether two ranges share a byte.  Two views of one buffer may take different columns of
// it: modulo the greatest common divisor g of the strides every row of x lies at the same
// place, and so does every row of y; where these places are apart no byte is shared.  Of
// equal strides, or where one range is a single piece, this decides exactly; of others
// the ranges count as overlapping when their ends do.
inline bool overlap(const Range& x, const Range& y) {
    if (!x.p || !y.p || !x.rows || !y.rows || !x.width || !y.width) return false;
    const uint64_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    if (a >= b + (y.rows - 1) * y.stride + y.width || b >= a + (x.rows - 1) * x.stride + x.width) return false;
    const uint64_t g = std::gcd(x.stride, y.stride);
    if (g == 0) return true;
    const uint64_t at = a <= b ? (b - a) % g : (g - (a - b) % g) % g;      // y's place, x at 0
    return at < x.width || at + y.width > g;
}

// No written range may overlap another.
template <size_t N>
int check_overlap(const Range (&r)[N]) {
    for (size_t i = 0; i < N; ++i)
        for (size_t j = i + 1; j < N; ++j)
            if ((r[i].written || r[j].written) && overlap(r[i], r[j]))
                return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s overlaps %s", r[i].what, r[j].what);
    return MOE_NVFP4_OK;
}

// rows x width elements at p (of no rows, nothing is looked at).
inline int check_rows(const char* what, const void* p, int64_t rows, int64_t width, int64_t stride, int dtype) {
    if (rows == 0 || width == 0) return MOE_NVFP4_OK;
    if (!p) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s is NULL", what);
    if (misaligned(p, moe::dtype_bytes(dtype)))
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s is not aligned to its elements", what);
    if (rows > 1 && stride < width)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s: row stride %lld < width %lld", what, (long long)stride,
                    (long long)width);
    if (rows > 1 && stride > (1LL << 40) / rows)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: %lld rows of stride %lld", what, (long long)rows,
                    (long long)stride);
    return MOE_NVFP4_OK;
}

inline int check_i32(const char* what, const void* p, bool optional) {
    if (!p && !optional) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s is NULL", what);
    if (misaligned(p, 4)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s must be 4-byte aligned", what);
    return MOE_NVFP4_OK;
}

inline int check_float_dtype(int dtype) {
    if (dtype != MOE_BF16 && dtype != MOE_F16 && dtype != MOE_F32)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "dtype %d is not bf16, f16 or f32", dtype);
    return MOE_NVFP4_OK;
}

inline int check_product(const moe_product_problem* p, const uint8_t* w, const uint8_t* w_scales, const int32_t* offsets) {
    if (!p) return fail(MOE_NVFP4_ERR_INVALID_ARG, "problem is NULL");
    if (p->rows < 0 || p->rows > (1 << 27)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "rows %d outside 0..2^27", p->rows);
    if (p->n < 1 || p->n > 65536) return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "n %d outside 1..65536", p->n);
    if (p->k < 32 || p->k > 65536 || p->k % 32)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "k %d: need a multiple of 32 in 32..65536", p->k);
    if (p->groups < 1 || p->groups > 1024)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "groups %d outside 1..1024", p->groups);
    if (!w || !w_scales) return fail(MOE_NVFP4_ERR_INVALID_ARG, "weights are NULL");
    if (misaligned(w, 16)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "weight codes must be 16-byte aligned");
    if (!offsets && p->groups != 1) return fail(MOE_NVFP4_ERR_INVALID_ARG, "offsets is NULL with %d groups", p->groups);
    return check_i32("offsets", offsets, true);
}

}  // namespace checks
}  // namespace moe
