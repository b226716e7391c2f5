// Host side of the operators declared in include/moe_ops.h: validation, the
// workspace plan of the dispatch, launches.
#include "../../include/moe_ops.h"

#include <hip/hip_runtime.h>

#include <numeric>

#include "kernels.h"
#include "ops.h"
#include "status.h"

namespace {

using moe::cu_count;
using moe::current_arch_ok;
using moe::fail;
using moe::hip_status;
using moe::ok;

bool misaligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Device memory that a call reads or writes: `rows` pieces of `width` bytes, `stride`
// bytes apart (nothing when p is NULL or a count is 0).
struct Range {
    const char* what;
    const void* p;
    uint64_t rows, width, stride;
    bool written;
};

Range dense(const char* what, const void* p, uint64_t bytes, bool written) {
    return Range{what, p, 1, bytes, 0, written};
}

// rows x width elements with a row stride (of one row, the stride is not looked at).
Range strided(const char* what, const void* p, int64_t rows, int64_t width, int64_t stride, int elem, bool written) {
    return Range{what, p, (uint64_t)rows, (uint64_t)(width * elem), rows > 1 ? (uint64_t)(stride * elem) : 0, written};
}

// Whether two ranges share a byte.  Two views of one buffer may take different columns of
// it: modulo the greatest common divisor g of the strides every row of x lies at the same
// place, and so does every row of y; where these places are apart no byte is shared.  Of
// equal strides, or where one range is a single piece, this decides exactly; of others
// the ranges count as overlapping when their ends do.
bool overlap(const Range& x, const Range& y) {
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
int check_rows(const char* what, const void* p, int64_t rows, int64_t width, int64_t stride, int dtype) {
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

int check_i32(const char* what, const void* p, bool optional) {
    if (!p && !optional) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s is NULL", what);
    if (misaligned(p, 4)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s must be 4-byte aligned", what);
    return MOE_NVFP4_OK;
}

int check_float_dtype(int dtype) {
    if (dtype != MOE_BF16 && dtype != MOE_F16 && dtype != MOE_F32)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "dtype %d is not bf16, f16 or f32", dtype);
    return MOE_NVFP4_OK;
}

int check_dispatch(const moe_dispatch_problem* p) {
    if (!p) return fail(MOE_NVFP4_ERR_INVALID_ARG, "problem is NULL");
    if (p->num_tokens < 0) return fail(MOE_NVFP4_ERR_INVALID_ARG, "num_tokens < 0");
    if (p->top_k < 1 || p->top_k > 32) return fail(MOE_NVFP4_ERR_INVALID_ARG, "top_k %d outside 1..32", p->top_k);
    if (p->num_experts < 1 || p->num_experts > 1024)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "num_experts %d outside 1..1024", p->num_experts);
    if (p->num_local_experts < 1) return fail(MOE_NVFP4_ERR_INVALID_ARG, "num_local_experts < 1");
    if (p->local_expert_offset < 0) return fail(MOE_NVFP4_ERR_INVALID_ARG, "local_expert_offset < 0");
    if ((long long)p->local_expert_offset + p->num_local_experts > p->num_experts)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "local_expert_offset + num_local_experts > num_experts");
    if (p->width < 1 || p->width > 65536)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "width %d outside 1..65536", p->width);
    if (p->dtype < MOE_BF16 || p->dtype > MOE_U8)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "unknown dtype %d", p->dtype);
    // pair numbers stay within int32
    if ((long long)p->num_tokens * p->top_k > (1LL << 27))
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "num_tokens * top_k > 2^27");
    return MOE_NVFP4_OK;
}

size_t dispatch_workspace(const moe_dispatch_problem& p) {
    if (p.num_tokens == 0) return 0;
    const moe::DispatchPlan d = moe::dispatch_plan(p.num_tokens, p.top_k);
    return d.one_launch ? 0 : (size_t)p.num_local_experts * ((size_t)d.blocks + 1) * 4;
}

int64_t pairs(const moe_dispatch_problem* p) { return (int64_t)p->num_tokens * p->top_k; }

// Rows, gradient rows, indices and weights of the combining calls share these checks.
int combine_rows(const moe_dispatch_problem* p, const int32_t* inv, const float* weights, bool weighted,
                 const void* rows, int64_t rows_stride, void* out, int64_t out_stride, void* stream) {
    int st = check_dispatch(p);
    if (st) return st;
    if ((st = check_float_dtype(p->dtype))) return st;
    const bool none = p->num_tokens == 0;
    if ((st = check_i32("inv", inv, none)) || (weighted && (st = check_i32("weights", weights, none)))) return st;
    if ((st = check_rows("rows", rows, pairs(p), p->width, rows_stride, p->dtype)) ||
        (st = check_rows("out", out, p->num_tokens, p->width, out_stride, p->dtype)))
        return st;
    const int eb = moe::dtype_bytes(p->dtype);
    const Range r[] = {strided("out", out, p->num_tokens, p->width, out_stride, eb, true),
                       strided("rows", rows, pairs(p), p->width, rows_stride, eb, false),
                       dense("inv", inv, pairs(p) * 4, false), dense("weights", weights, pairs(p) * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (p->num_tokens == 0) return ok();
    moe::CombineRowsArgs a{};
    a.T = p->num_tokens; a.k = p->top_k; a.d = p->width; a.dtype = p->dtype;
    a.inv = inv; a.w = weighted ? weights : nullptr;
    a.rows = rows; a.rs = rows_stride; a.out = out; a.os = out_stride;
    st = hip_status(moe::launch_combine_rows(a, static_cast<hipStream_t>(stream)), "combine launch");
    return st ? st : ok();
}

int check_product(const moe_product_problem* p, const uint8_t* w, const uint8_t* w_scales, const int32_t* offsets) {
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

moe::ProductArgs product_args(const moe_product_problem* p, const void* a, int64_t as, const uint8_t* w,
                              const uint8_t* w_scales, const int32_t* offsets, void* out, int out_dtype, int64_t os) {
    moe::ProductArgs g{};
    g.M = p->rows; g.N = p->n; g.K = p->k; g.G = p->groups;
    g.a = a; g.as = as; g.w = w; g.w_s = w_scales; g.offsets = offsets;
    g.out = out; g.out_dtype = out_dtype; g.os = os;
    return g;
}

}  // namespace

extern "C" {

int moe_dispatch_workspace_size(const moe_dispatch_problem* p, size_t* bytes) {
    if (!bytes) return fail(MOE_NVFP4_ERR_INVALID_ARG, "bytes is NULL");
    const int st = check_dispatch(p);
    if (st) return st;
    *bytes = dispatch_workspace(*p);
    return ok();
}

int moe_dispatch(const moe_dispatch_problem* p, const int32_t* ids, const void* x, int64_t x_stride, int32_t* counts,
                 int32_t* offsets, int32_t* perm, int32_t* inv, void* rows, int64_t rows_stride, void* workspace,
                 size_t workspace_bytes, void* stream) {
    int st = check_dispatch(p);
    if (st) return st;
    const bool none = p->num_tokens == 0;
    if ((st = check_i32("ids", ids, none)) || (st = check_i32("counts", counts, true)) ||
        (st = check_i32("offsets", offsets, true)) || (st = check_i32("perm", perm, true)) ||
        (st = check_i32("inv", inv, true)))
        return st;
    if (!none && !x != !rows) return fail(MOE_NVFP4_ERR_INVALID_ARG, "x and rows must be given together");
    if (x && ((st = check_rows("x", x, p->num_tokens, p->width, x_stride, p->dtype)) ||
              (st = check_rows("rows", rows, pairs(p), p->width, rows_stride, p->dtype))))
        return st;
    const size_t need = dispatch_workspace(*p);
    if (workspace_bytes < need)
        return fail(MOE_NVFP4_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < required %zu", workspace_bytes, need);
    if (need && !workspace) return fail(MOE_NVFP4_ERR_INVALID_ARG, "workspace is NULL");
    if (need && misaligned(workspace, 4)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
    const int eb = moe::dtype_bytes(p->dtype);
    const size_t np = (size_t)pairs(p), L = (size_t)p->num_local_experts;
    const Range r[] = {strided("rows", rows, pairs(p), p->width, rows_stride, eb, true),
                       dense("counts", counts, L * 4, true),
                       dense("offsets", offsets, (L + 1) * 4, true),
                       dense("perm", perm, np * 4, true),
                       dense("inv", inv, np * 4, true),
                       dense("workspace", workspace, need, true),
                       strided("x", x, p->num_tokens, p->width, x_stride, eb, false),
                       dense("ids", ids, np * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (p->num_tokens == 0) {
        // no pair: counts and offsets are still written
        if ((counts && (st = hip_status(moe::launch_fill_u32(reinterpret_cast<uint32_t*>(counts), L, 0u, s), "fill"))) ||
            (offsets &&
             (st = hip_status(moe::launch_fill_u32(reinterpret_cast<uint32_t*>(offsets), L + 1, 0u, s), "fill"))))
            return st;
        return ok();
    }
    moe::DispatchArgs a{};
    a.T = p->num_tokens; a.k = p->top_k; a.L = p->num_local_experts; a.offset = p->local_expert_offset;
    a.d = p->width; a.dtype = p->dtype;
    a.ids = ids; a.x = x; a.xs = x_stride; a.counts = counts; a.offsets = offsets; a.perm = perm; a.inv = inv;
    a.rows = rows; a.rs = rows_stride;
    if (need) {
        a.totals = static_cast<int32_t*>(workspace);
        a.block_counts = a.totals + L;
    }
    st = hip_status(moe::launch_dispatch(a, s), "dispatch launch");
    return st ? st : ok();
}

int moe_dispatch_backward(const moe_dispatch_problem* p, const int32_t* inv, const void* drows, int64_t drows_stride,
                          void* dx, int64_t dx_stride, void* stream) {
    return combine_rows(p, inv, nullptr, false, drows, drows_stride, dx, dx_stride, stream);
}

int moe_combine(const moe_dispatch_problem* p, const int32_t* inv, const float* weights, const void* rows,
                int64_t rows_stride, void* out, int64_t out_stride, void* stream) {
    return combine_rows(p, inv, weights, true, rows, rows_stride, out, out_stride, stream);
}

int moe_combine_backward(const moe_dispatch_problem* p, const int32_t* inv, const float* weights, const void* rows,
                         int64_t rows_stride, const void* dout, int64_t dout_stride, void* drows,
                         int64_t drows_stride, float* dweights, void* stream) {
    int st = check_dispatch(p);
    if (st) return st;
    if ((st = check_float_dtype(p->dtype))) return st;
    const bool none = p->num_tokens == 0;
    if ((st = check_i32("inv", inv, none)) || (st = check_i32("weights", weights, none)) ||
        (st = check_i32("dweights", dweights, true)))
        return st;
    if ((st = check_rows("dout", dout, p->num_tokens, p->width, dout_stride, p->dtype))) return st;
    if (dweights && (st = check_rows("rows", rows, pairs(p), p->width, rows_stride, p->dtype))) return st;
    if (drows && (st = check_rows("drows", drows, pairs(p), p->width, drows_stride, p->dtype))) return st;
    const int eb = moe::dtype_bytes(p->dtype);
    const size_t pb = (size_t)pairs(p) * 4;
    const Range r[] = {strided("drows", drows, pairs(p), p->width, drows_stride, eb, true),
                       dense("dweights", dweights, pb, true),
                       strided("rows", dweights ? rows : nullptr, pairs(p), p->width, rows_stride, eb, false),
                       strided("dout", dout, p->num_tokens, p->width, dout_stride, eb, false),
                       dense("inv", inv, pb, false),
                       dense("weights", weights, pb, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (p->num_tokens == 0 || (!drows && !dweights)) return ok();
    moe::CombineGradArgs a{};
    a.T = p->num_tokens; a.k = p->top_k; a.d = p->width; a.dtype = p->dtype;
    a.inv = inv; a.w = weights; a.rows = dweights ? rows : nullptr; a.rs = rows_stride;
    a.dout = dout; a.dos = dout_stride; a.drows = drows; a.drs = drows_stride; a.dw = dweights;
    st = hip_status(moe::launch_combine_grad(a, static_cast<hipStream_t>(stream)), "combine gradient launch");
    return st ? st : ok();
}

static int check_mxfp4_tensor(int64_t R, int32_t C, const uint8_t* codes, const uint8_t* scales) {
    if (R < 0 || C < 0) return fail(MOE_NVFP4_ERR_INVALID_ARG, "negative size");
    if (C % 32) return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "C %d is not a multiple of 32", C);
    if (C > 0 && R > (1LL << 40) / C) return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "tensor too large");
    if (R == 0 || C == 0) return MOE_NVFP4_OK;
    if (!codes || !scales) return fail(MOE_NVFP4_ERR_INVALID_ARG, "codes/scales is NULL");
    if (misaligned(codes, 16)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "codes must be 16-byte aligned");
    return MOE_NVFP4_OK;
}

int moe_mxfp4_quantize(const void* x, int32_t dtype, int64_t R, int32_t C, int64_t x_stride, uint8_t* codes,
                       uint8_t* scales, void* stream) {
    int st = check_float_dtype(dtype);
    if (st) return st;
    if ((st = check_mxfp4_tensor(R, C, codes, scales))) return st;
    if ((st = check_rows("x", x, R, C, x_stride, dtype))) return st;
    const Range r[] = {dense("codes", codes, (size_t)R * C / 2, true),
                       dense("scales", scales, (size_t)R * C / 32, true),
                       strided("x", x, R, C, x_stride, moe::dtype_bytes(dtype), false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (R == 0 || C == 0) return ok();
    st = hip_status(moe::launch_mxfp4_quantize(x, dtype, R, C, x_stride, codes, scales, static_cast<hipStream_t>(stream)),
                    "MXFP4 quantizer launch");
    return st ? st : ok();
}

int moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int32_t C, int32_t dtype, void* out,
                         int64_t out_stride, void* stream) {
    int st = check_float_dtype(dtype);
    if (st) return st;
    if ((st = check_mxfp4_tensor(R, C, codes, scales))) return st;
    if ((st = check_rows("out", out, R, C, out_stride, dtype))) return st;
    const Range r[] = {strided("out", out, R, C, out_stride, moe::dtype_bytes(dtype), true),
                       dense("codes", codes, (size_t)R * C / 2, false),
                       dense("scales", scales, (size_t)R * C / 32, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (R == 0 || C == 0) return ok();
    st = hip_status(moe::launch_mxfp4_dequantize(codes, scales, R, C, dtype, out, out_stride,
                                                 static_cast<hipStream_t>(stream)),
                    "MXFP4 dequantizer launch");
    return st ? st : ok();
}

int moe_mxfp4_product(const moe_product_problem* p, const void* a, const uint8_t* a_scales, int64_t a_stride,
                      const uint8_t* w, const uint8_t* w_scales, const int32_t* offsets, void* out, int32_t out_dtype,
                      int64_t out_stride, void* stream) {
    int st = check_product(p, w, w_scales, offsets);
    if (st) return st;
    if ((st = check_float_dtype(out_dtype))) return st;
    const int64_t M = p->rows, N = p->n, K = p->k;
    if (a_scales) {
        a_stride = K;                                     // dense
        if (!a && M > 0) return fail(MOE_NVFP4_ERR_INVALID_ARG, "a is NULL");
    } else {
        if ((st = check_rows("a", a, M, K, a_stride, MOE_BF16))) return st;
        if (M > 1 && a_stride % 8)
            return fail(MOE_NVFP4_ERR_INVALID_ARG, "a: row stride %lld is not a multiple of 8", (long long)a_stride);
    }
    if (misaligned(a, 16)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "a must be 16-byte aligned");
    if ((st = check_rows("out", out, M, N, out_stride, out_dtype))) return st;
    const size_t wn = (size_t)p->groups * N;
    const Range r[] = {strided("out", out, M, N, out_stride, moe::dtype_bytes(out_dtype), true),
                       a_scales ? dense("a", a, (size_t)M * K / 2, false) : strided("a", a, M, K, a_stride, 2, false),
                       dense("a_scales", a_scales, (size_t)M * K / 32, false),
                       dense("w", w, wn * K / 2, false),
                       dense("w_scales", w_scales, wn * K / 32, false),
                       dense("offsets", offsets, ((size_t)p->groups + 1) * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev, cus;
    if ((st = current_arch_ok(&dev))) return st;
    if (M == 0) return ok();
    if ((st = cu_count(dev, &cus))) return st;
    moe::ProductArgs g = product_args(p, a, a_stride, w, w_scales, offsets, out, out_dtype, out_stride);
    g.a_s = a_scales;
    st = hip_status(moe::launch_product(g, cus, static_cast<hipStream_t>(stream)), "MXFP4 product launch");
    return st ? st : ok();
}

int moe_mxfp4_product_backward(const moe_product_problem* p, const void* dout, int64_t dout_stride, const uint8_t* w,
                               const uint8_t* w_scales, const int32_t* offsets, void* drows, int32_t drows_dtype,
                               int64_t drows_stride, void* stream) {
    int st = check_product(p, w, w_scales, offsets);
    if (st) return st;
    if ((st = check_float_dtype(drows_dtype))) return st;
    const int64_t M = p->rows, N = p->n, K = p->k;
    if ((st = check_rows("dout", dout, M, N, dout_stride, MOE_BF16)) ||
        (st = check_rows("drows", drows, M, K, drows_stride, drows_dtype)))
        return st;
    const size_t wn = (size_t)p->groups * N;
    const Range r[] = {strided("drows", drows, M, K, drows_stride, moe::dtype_bytes(drows_dtype), true),
                       strided("dout", dout, M, N, dout_stride, 2, false),
                       dense("w", w, wn * K / 2, false),
                       dense("w_scales", w_scales, wn * K / 32, false),
                       dense("offsets", offsets, ((size_t)p->groups + 1) * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev, cus;
    if ((st = current_arch_ok(&dev))) return st;
    if (M == 0) return ok();
    if ((st = cu_count(dev, &cus))) return st;
    const moe::ProductArgs g = product_args(p, dout, dout_stride, w, w_scales, offsets, drows, drows_dtype, drows_stride);
    st = hip_status(moe::launch_product_grad(g, cus, static_cast<hipStream_t>(stream)), "MXFP4 product gradient launch");
    return st ? st : ok();
}

}  // extern "C"
