// Internal interface between the host code of include/moe_block.h (block.cpp) and its
// gfx950 kernels (topk.hip, norm.hip, swiglu.hip, mxfp8.hip; the product: product.hip, product8.hip).  Strides are in
// elements.
#pragma once
#include "ops.h"

namespace moe {

struct RouteArgs {
    int T, E, k, dtype;
    int sigmoid, groups, top_groups, group_keys, renormalize;
    float scale;
    const void* logits;           // [T][E]
    int64_t ls;
    const float* bias;            // [E] or nullptr
    int32_t* ids;                 // [T][k]
    float* w;                     // [T][k]
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct RouteGradArgs {
    int T, E, k, dtype;
    int sigmoid, renormalize;
    float scale;
    const void* logits;           // [T][E]
    int64_t ls;
    const int32_t* ids;           // [T][k]
    const float* dw;              // [T][k]
    void* dlogits;                // [T][E]
    int64_t ds;
};
hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t s);

struct NormArgs {
    int T, d, dtype, wdtype;
    float eps;
    const void* x;                // [T][d]
    int64_t xs;
    const void* res;              // [T][d] or nullptr
    int64_t ress;
    const void* w;                // [d]
    void* h;                      // [T][d] or nullptr
    int64_t hs;
    void* y;                      // [T][d] or nullptr
    int64_t ys;
    uint8_t* codes;               // [T][d] or nullptr
    uint8_t* scales;              // [T][d/32]
    float* rstd;                  // [T] or nullptr
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
    int T, d, dtype, wdtype;
    const void* h;                // [T][d]
    int64_t hs;
    const void* w;                // [d]
    const float* rstd;            // [T]
    const void* dy;               // [T][d]
    int64_t dys;
    const void* dh;               // [T][d] or nullptr
    int64_t dhs;
    void* dx;                     // [T][d] or nullptr
    int64_t dxs;
    float* dw;                    // [d] or nullptr
    float* partial;               // workspace [norm_grad_blocks][d]
};
int norm_grad_blocks(int T, int d);          // rows of partial sums
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s);

struct SwigluArgs {
    int M, F, G, dtype;
    const int32_t* offsets;       // [G+1] or nullptr
    const void* u;                // [M][2F]; backward: or MXFP8 codes [M][2F]
    int64_t us;
    void* a;                      // [M][F] or nullptr; backward: da
    int64_t as;
    uint8_t* codes;               // [M][F] or nullptr
    uint8_t* scales;              // [M][F/32]
    uint8_t* kept;                // [M][2F] or nullptr
    uint8_t* kept_s;              // [M][2F/32]; backward: nullptr: u is of dtype
    void* du;                     // backward: [M][2F]
    int64_t dus;
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);
hipError_t launch_swiglu_grad(const SwigluArgs& a, hipStream_t s);

hipError_t launch_mxfp8_quantize(const void* x, int dtype, int64_t R, int C, int64_t xs, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s);
hipError_t launch_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int C, int dtype,
                                   void* out, int64_t os, hipStream_t s);

}  // namespace moe
