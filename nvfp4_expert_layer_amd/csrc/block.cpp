// Host side of the operators declared in include/moe_block.h: validation, launches.
#include "../../include/moe_block.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "block.h"
#include "checks.h"
#include "status.h"

namespace {

using namespace moe::checks;
using moe::cu_count;
using moe::current_arch_ok;
using moe::dtype_bytes;
using moe::fail;
using moe::hip_status;
using moe::ok;

int check_route(const moe_route_problem* p) {
    if (!p) return fail(MOE_NVFP4_ERR_INVALID_ARG, "problem is NULL");
    if (p->num_tokens < 0) return fail(MOE_NVFP4_ERR_INVALID_ARG, "num_tokens < 0");
    if (p->num_experts < 1 || p->num_experts > 1024)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "num_experts %d outside 1..1024", p->num_experts);
    if (p->scores != MOE_ROUTE_SOFTMAX && p->scores != MOE_ROUTE_SIGMOID)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "unknown scores %d", p->scores);
    if (p->num_groups < 1 || p->num_groups > 64)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "num_groups %d outside 1..64", p->num_groups);
    if (p->num_experts % p->num_groups)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "num_groups %d does not divide num_experts %d", p->num_groups,
                    p->num_experts);
    if (p->top_groups < 1 || p->top_groups > p->num_groups)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "top_groups %d outside 1..num_groups", p->top_groups);
    if (p->group_keys < 1 || p->group_keys > 2)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "group_keys %d is not 1 or 2", p->group_keys);
    if (p->top_k < 1 || p->top_k > 32) return fail(MOE_NVFP4_ERR_INVALID_ARG, "top_k %d outside 1..32", p->top_k);
    if (p->top_k > p->top_groups * (p->num_experts / p->num_groups))
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "top_k %d > the experts of top_groups groups", p->top_k);
    if (p->renormalize != 0 && p->renormalize != 1)
        return fail(MOE_NVFP4_ERR_INVALID_ARG, "renormalize %d is not 0 or 1", p->renormalize);
    if (!std::isfinite(p->scale)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "scale is not finite");
    if ((long long)p->num_tokens * p->top_k > (1LL << 27))
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "num_tokens * top_k > 2^27");
    return check_float_dtype(p->dtype);
}

int check_norm(const moe_norm_problem* p) {
    if (!p) return fail(MOE_NVFP4_ERR_INVALID_ARG, "problem is NULL");
    if (p->rows < 0 || p->rows > (1 << 27)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "rows %d outside 0..2^27", p->rows);
    if (p->width < 1 || p->width > 65536)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "width %d outside 1..65536", p->width);
    if (!std::isfinite(p->eps) || p->eps < 0.f) return fail(MOE_NVFP4_ERR_INVALID_ARG, "eps is not finite and >= 0");
    const int st = check_float_dtype(p->dtype);
    return st ? st : check_float_dtype(p->weight_dtype);
}

int check_swiglu(const moe_swiglu_problem* p, const int32_t* offsets) {
    if (!p) return fail(MOE_NVFP4_ERR_INVALID_ARG, "problem is NULL");
    if (p->rows < 0 || p->rows > (1 << 27)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "rows %d outside 0..2^27", p->rows);
    if (p->width < 1 || p->width > 65536)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "width %d outside 1..65536", p->width);
    if (p->groups < 1 || p->groups > 1024)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "groups %d outside 1..1024", p->groups);
    const int st = check_float_dtype(p->dtype);
    return st ? st : check_i32("offsets", offsets, true);
}

// Codes and scales of an MXFP8 tensor of `rows` rows of `width` elements: both or neither.
int check_mx(const char* what, const void* codes, const void* scales, int64_t rows, int64_t width) {
    if (rows == 0 || (!codes && !scales)) return MOE_NVFP4_OK;
    if (!codes || !scales) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s: codes and scales must be given together", what);
    if (width % 32)
        return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: width %lld is not a multiple of 32", what, (long long)width);
    if (misaligned(codes, 16)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
    return MOE_NVFP4_OK;
}

int check_f32(const char* what, const void* p, bool optional) { return check_i32(what, p, optional); }

int check_mx_tensor(int64_t R, int32_t C, const uint8_t* codes, const uint8_t* scales) {
    if (R < 0 || C < 0) return fail(MOE_NVFP4_ERR_INVALID_ARG, "negative size");
    if (C % 32) return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "C %d is not a multiple of 32", C);
    if (C > 0 && R > (1LL << 40) / C) return fail(MOE_NVFP4_ERR_UNSUPPORTED_SHAPE, "tensor too large");
    if (R == 0 || C == 0) return MOE_NVFP4_OK;
    if (!codes || !scales) return fail(MOE_NVFP4_ERR_INVALID_ARG, "codes/scales is NULL");
    return check_mx("codes", codes, scales, R, C);
}

}  // namespace

extern "C" {

int moe_route(const moe_route_problem* p, const void* logits, int64_t logits_stride, const float* bias, int32_t* ids,
              float* weights, void* stream) {
    int st = check_route(p);
    if (st) return st;
    const bool none = p->num_tokens == 0;
    const int64_t T = p->num_tokens, E = p->num_experts, pairs = T * p->top_k;
    if ((st = check_rows("logits", logits, T, E, logits_stride, p->dtype)) || (st = check_f32("bias", bias, true)) ||
        (st = check_i32("ids", ids, none)) || (st = check_f32("weights", weights, none)))
        return st;
    const Range r[] = {dense("ids", ids, pairs * 4, true), dense("weights", weights, pairs * 4, true),
                       strided("logits", logits, T, E, logits_stride, dtype_bytes(p->dtype), false),
                       dense("bias", bias, none ? 0 : E * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (none) return ok();
    moe::RouteArgs a{};
    a.T = p->num_tokens; a.E = p->num_experts; a.k = p->top_k; a.dtype = p->dtype;
    a.sigmoid = p->scores == MOE_ROUTE_SIGMOID; a.groups = p->num_groups; a.top_groups = p->top_groups;
    a.group_keys = p->group_keys; a.renormalize = p->renormalize; a.scale = p->scale;
    a.logits = logits; a.ls = logits_stride; a.bias = bias; a.ids = ids; a.w = weights;
    st = hip_status(moe::launch_route(a, static_cast<hipStream_t>(stream)), "route launch");
    return st ? st : ok();
}

int moe_route_backward(const moe_route_problem* p, const void* logits, int64_t logits_stride, const int32_t* ids,
                       const float* dweights, void* dlogits, int64_t dlogits_stride, void* stream) {
    int st = check_route(p);
    if (st) return st;
    const bool none = p->num_tokens == 0;
    const int64_t T = p->num_tokens, E = p->num_experts, pairs = T * p->top_k;
    if ((st = check_rows("logits", logits, T, E, logits_stride, p->dtype)) || (st = check_i32("ids", ids, none)) ||
        (st = check_f32("dweights", dweights, none)) ||
        (st = check_rows("dlogits", dlogits, T, E, dlogits_stride, p->dtype)))
        return st;
    const int eb = dtype_bytes(p->dtype);
    const Range r[] = {strided("dlogits", dlogits, T, E, dlogits_stride, eb, true),
                       strided("logits", logits, T, E, logits_stride, eb, false),
                       dense("ids", ids, pairs * 4, false), dense("dweights", dweights, pairs * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (none) return ok();
    moe::RouteGradArgs a{};
    a.T = p->num_tokens; a.E = p->num_experts; a.k = p->top_k; a.dtype = p->dtype;
    a.sigmoid = p->scores == MOE_ROUTE_SIGMOID; a.renormalize = p->renormalize; a.scale = p->scale;
    a.logits = logits; a.ls = logits_stride; a.ids = ids; a.dw = dweights; a.dlogits = dlogits; a.ds = dlogits_stride;
    st = hip_status(moe::launch_route_grad(a, static_cast<hipStream_t>(stream)), "route gradient launch");
    return st ? st : ok();
}

int moe_norm(const moe_norm_problem* p, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
             const void* weight, void* h, int64_t h_stride, void* y, int64_t y_stride, uint8_t* codes, uint8_t* scales,
             float* rstd, void* stream) {
    int st = check_norm(p);
    if (st) return st;
    const int64_t T = p->rows, d = p->width;
    if ((st = check_rows("x", x, T, d, x_stride, p->dtype)) ||
        (residual && (st = check_rows("residual", residual, T, d, residual_stride, p->dtype))) ||
        (st = check_rows("weight", weight, T > 0 ? 1 : 0, d, d, p->weight_dtype)) ||
        (h && (st = check_rows("h", h, T, d, h_stride, p->dtype))) ||
        (y && (st = check_rows("y", y, T, d, y_stride, p->dtype))) || (st = check_mx("codes", codes, scales, T, d)) ||
        (st = check_f32("rstd", rstd, true)))
        return st;
    const int eb = dtype_bytes(p->dtype);
    const Range r[] = {strided("h", h, T, d, h_stride, eb, true),
                       strided("y", y, T, d, y_stride, eb, true),
                       dense("codes", codes, T * d, true),
                       dense("scales", scales, T * (d / 32), true),
                       dense("rstd", rstd, T * 4, true),
                       strided("x", x, T, d, x_stride, eb, false),
                       strided("residual", residual, T, d, residual_stride, eb, false),
                       dense("weight", weight, T > 0 ? d * dtype_bytes(p->weight_dtype) : 0, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (T == 0 || (!h && !y && !codes && !rstd)) return ok();
    moe::NormArgs a{};
    a.T = p->rows; a.d = p->width; a.dtype = p->dtype; a.wdtype = p->weight_dtype; a.eps = p->eps;
    a.x = x; a.xs = x_stride; a.res = residual; a.ress = residual_stride; a.w = weight; a.h = h; a.hs = h_stride;
    a.y = y; a.ys = y_stride; a.codes = codes; a.scales = scales; a.rstd = rstd;
    st = hip_status(moe::launch_norm(a, static_cast<hipStream_t>(stream)), "norm launch");
    return st ? st : ok();
}

int moe_norm_workspace_size(const moe_norm_problem* p, size_t* bytes) {
    if (!bytes) return fail(MOE_NVFP4_ERR_INVALID_ARG, "bytes is NULL");
    const int st = check_norm(p);
    if (st) return st;
    *bytes = (size_t)moe::norm_grad_blocks(p->rows, p->width) * p->width * 4;
    return ok();
}

int moe_norm_backward(const moe_norm_problem* p, const void* h, int64_t h_stride, const void* weight,
                      const float* rstd, const void* dy, int64_t dy_stride, const void* dh, int64_t dh_stride, void* dx,
                      int64_t dx_stride, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_norm(p);
    if (st) return st;
    const int64_t T = p->rows, d = p->width;
    if ((st = check_rows("h", h, T, d, h_stride, p->dtype)) || (st = check_f32("rstd", rstd, T == 0)) ||
        (st = check_rows("dy", dy, T, d, dy_stride, p->dtype)) ||
        (dx && (st = check_rows("weight", weight, T > 0 ? 1 : 0, d, d, p->weight_dtype))) ||
        (dx && dh && (st = check_rows("dh", dh, T, d, dh_stride, p->dtype))) ||
        (dx && (st = check_rows("dx", dx, T, d, dx_stride, p->dtype))) || (st = check_f32("dweight", dweight, true)))
        return st;
    const size_t need = dweight ? (size_t)moe::norm_grad_blocks(p->rows, p->width) * d * 4 : 0;
    if (workspace_bytes < need)
        return fail(MOE_NVFP4_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < required %zu", workspace_bytes, need);
    if (need && !workspace) return fail(MOE_NVFP4_ERR_INVALID_ARG, "workspace is NULL");
    if (need && misaligned(workspace, 4)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
    const int eb = dtype_bytes(p->dtype);
    const Range r[] = {strided("dx", dx, T, d, dx_stride, eb, true),
                       dense("dweight", dweight, d * 4, true),
                       dense("workspace", workspace, need, true),
                       strided("h", h, T, d, h_stride, eb, false),
                       dense("weight", dx ? weight : nullptr, T > 0 ? d * dtype_bytes(p->weight_dtype) : 0, false),
                       dense("rstd", rstd, T * 4, false),
                       strided("dy", dy, T, d, dy_stride, eb, false),
                       strided("dh", dx ? dh : nullptr, T, d, dh_stride, eb, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (!dx && !dweight) return ok();
    moe::NormGradArgs a{};
    a.T = p->rows; a.d = p->width; a.dtype = p->dtype; a.wdtype = p->weight_dtype;
    a.h = h; a.hs = h_stride; a.w = weight; a.rstd = rstd; a.dy = dy; a.dys = dy_stride; a.dh = dx ? dh : nullptr;
    a.dhs = dh_stride; a.dx = dx; a.dxs = dx_stride; a.dw = dweight; a.partial = static_cast<float*>(workspace);
    st = hip_status(moe::launch_norm_grad(a, static_cast<hipStream_t>(stream)), "norm gradient launch");
    return st ? st : ok();
}

int moe_swiglu(const moe_swiglu_problem* p, const void* u, int64_t u_stride, const int32_t* offsets, void* a,
               int64_t a_stride, uint8_t* codes, uint8_t* scales, uint8_t* kept, uint8_t* kept_scales, void* stream) {
    int st = check_swiglu(p, offsets);
    if (st) return st;
    const int64_t M = p->rows, F = p->width;
    if ((st = check_rows("u", u, M, 2 * F, u_stride, p->dtype)) ||
        (a && (st = check_rows("a", a, M, F, a_stride, p->dtype))) || (st = check_mx("codes", codes, scales, M, F)) ||
        (st = check_mx("kept", kept, kept_scales, M, F)))
        return st;
    const int eb = dtype_bytes(p->dtype);
    const Range r[] = {strided("a", a, M, F, a_stride, eb, true),
                       dense("codes", codes, M * F, true),
                       dense("scales", scales, M * (F / 32), true),
                       dense("kept", kept, M * 2 * F, true),
                       dense("kept_scales", kept_scales, M * 2 * (F / 32), true),
                       strided("u", u, M, 2 * F, u_stride, eb, false),
                       dense("offsets", offsets, ((size_t)p->groups + 1) * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (M == 0 || (!a && !codes && !kept)) return ok();
    moe::SwigluArgs s{};
    s.M = p->rows; s.F = p->width; s.G = p->groups; s.dtype = p->dtype; s.offsets = offsets;
    s.u = u; s.us = u_stride; s.a = a; s.as = a_stride; s.codes = codes; s.scales = scales; s.kept = kept;
    s.kept_s = kept_scales;
    st = hip_status(moe::launch_swiglu(s, static_cast<hipStream_t>(stream)), "SwiGLU launch");
    return st ? st : ok();
}

int moe_swiglu_backward(const moe_swiglu_problem* p, const void* u, int64_t u_stride, const uint8_t* kept_scales,
                        const int32_t* offsets, const void* da, int64_t da_stride, void* du, int64_t du_stride,
                        void* stream) {
    int st = check_swiglu(p, offsets);
    if (st) return st;
    const int64_t M = p->rows, F = p->width;
    if (kept_scales) {
        if ((st = check_mx("u", u, kept_scales, M, F))) return st;
    } else if ((st = check_rows("u", u, M, 2 * F, u_stride, p->dtype))) {
        return st;
    }
    if ((st = check_rows("da", da, M, F, da_stride, p->dtype)) ||
        (st = check_rows("du", du, M, 2 * F, du_stride, p->dtype)))
        return st;
    const int eb = dtype_bytes(p->dtype);
    const Range r[] = {strided("du", du, M, 2 * F, du_stride, eb, true),
                       kept_scales ? dense("u", u, M * 2 * F, false) : strided("u", u, M, 2 * F, u_stride, eb, false),
                       dense("kept_scales", kept_scales, M * 2 * (F / 32), false),
                       strided("da", da, M, F, da_stride, eb, false),
                       dense("offsets", offsets, ((size_t)p->groups + 1) * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (M == 0) return ok();
    moe::SwigluArgs s{};
    s.M = p->rows; s.F = p->width; s.G = p->groups; s.dtype = p->dtype; s.offsets = offsets;
    s.u = u; s.us = u_stride; s.kept_s = const_cast<uint8_t*>(kept_scales); s.a = const_cast<void*>(da); s.as = da_stride;
    s.du = du; s.dus = du_stride;
    st = hip_status(moe::launch_swiglu_grad(s, static_cast<hipStream_t>(stream)), "SwiGLU gradient launch");
    return st ? st : ok();
}

int moe_mxfp8_quantize(const void* x, int32_t dtype, int64_t R, int32_t C, int64_t x_stride, uint8_t* codes,
                       uint8_t* scales, void* stream) {
    int st = check_float_dtype(dtype);
    if (st) return st;
    if ((st = check_mx_tensor(R, C, codes, scales)) || (st = check_rows("x", x, R, C, x_stride, dtype))) return st;
    const Range r[] = {dense("codes", codes, (size_t)R * C, true), dense("scales", scales, (size_t)R * C / 32, true),
                       strided("x", x, R, C, x_stride, dtype_bytes(dtype), false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (R == 0 || C == 0) return ok();
    st = hip_status(moe::launch_mxfp8_quantize(x, dtype, R, C, x_stride, codes, scales, static_cast<hipStream_t>(stream)),
                    "MXFP8 quantizer launch");
    return st ? st : ok();
}

int moe_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int32_t C, int32_t dtype, void* out,
                         int64_t out_stride, void* stream) {
    int st = check_float_dtype(dtype);
    if (st) return st;
    if ((st = check_mx_tensor(R, C, codes, scales)) || (st = check_rows("out", out, R, C, out_stride, dtype))) return st;
    const Range r[] = {strided("out", out, R, C, out_stride, dtype_bytes(dtype), true),
                       dense("codes", codes, (size_t)R * C, false), dense("scales", scales, (size_t)R * C / 32, false)};
    if ((st = check_overlap(r))) return st;
    int dev;
    if ((st = current_arch_ok(&dev))) return st;
    if (R == 0 || C == 0) return ok();
    st = hip_status(moe::launch_mxfp8_dequantize(codes, scales, R, C, dtype, out, out_stride,
                                                 static_cast<hipStream_t>(stream)),
                    "MXFP8 dequantizer launch");
    return st ? st : ok();
}

int moe_mxfp8_product(const moe_product_problem* p, const uint8_t* a, const uint8_t* a_scales, const uint8_t* w,
                      const uint8_t* w_scales, const int32_t* offsets, void* out, int32_t out_dtype,
                      int64_t out_stride, void* stream) {
    int st = check_product(p, w, w_scales, offsets);
    if (st) return st;
    if ((st = check_float_dtype(out_dtype))) return st;
    const int64_t M = p->rows, N = p->n, K = p->k;
    if (M > 0 && (!a || !a_scales)) return fail(MOE_NVFP4_ERR_INVALID_ARG, "a is NULL");
    if ((st = check_mx("a", a, a_scales, M, K)) || (st = check_rows("out", out, M, N, out_stride, out_dtype))) return st;
    const size_t wn = (size_t)p->groups * N;
    const Range r[] = {strided("out", out, M, N, out_stride, dtype_bytes(out_dtype), true),
                       dense("a", a, (size_t)M * K, false),
                       dense("a_scales", a_scales, (size_t)M * K / 32, false),
                       dense("w", w, wn * K / 2, false),
                       dense("w_scales", w_scales, wn * K / 32, false),
                       dense("offsets", offsets, ((size_t)p->groups + 1) * 4, false)};
    if ((st = check_overlap(r))) return st;
    int dev, cus;
    if ((st = current_arch_ok(&dev))) return st;
    if (M == 0) return ok();
    if ((st = cu_count(dev, &cus))) return st;
    moe::ProductArgs g{};
    g.M = p->rows; g.N = p->n; g.K = p->k; g.G = p->groups;
    g.a = a; g.a_s = a_scales; g.a8 = true; g.as = K; g.w = w; g.w_s = w_scales; g.offsets = offsets;
    g.out = out; g.out_dtype = out_dtype; g.os = out_stride;
    st = hip_status(moe::launch_product(g, cus, static_cast<hipStream_t>(stream)), "MXFP8 product launch");
    return st ? st : ok();
}

}  // extern "C"
