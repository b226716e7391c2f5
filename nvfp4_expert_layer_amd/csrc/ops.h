// Internal interface between the operators' host code (ops.cpp) and their gfx950
// kernels (dispatch.hip, mxfp4.hip, product.hip).  Strides are in elements.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

// Four and two dwords at any byte address: global loads and stores of gfx950 need no
// alignment (the compiler keeps one instruction); rows of any stride use them.
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(1)));

namespace moe {

enum { kBF16 = 0, kF16 = 1, kF32 = 2, kU8 = 3 };       // moe_dtype
inline int dtype_bytes(int t) { return t == kF32 ? 4 : (t == kU8 ? 1 : 2); }

struct DispatchArgs {
    int T, k, L, offset, d, dtype;
    const int32_t* ids;           // [T][k]
    const void* x;                // [T][d], nullptr: the plan alone
    int64_t xs;
    int32_t *counts, *offsets, *perm, *inv;            // each may be nullptr
    void* rows;                   // [T*k][d]
    int64_t rs;
    int32_t* block_counts;        // workspace [L][blocks], large batches
    int32_t* totals;              // workspace [L], large batches
};
struct DispatchPlan {
    int tokens_per_block, blocks;
    bool one_launch;              // every block counts the pairs before its own by itself
};
DispatchPlan dispatch_plan(int T, int k);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s);

struct CombineRowsArgs {          // out[t] = sum_j w_tj rows[inv_tj]; w == nullptr: ones
    int T, k, d, dtype;
    const int32_t* inv;
    const float* w;
    const void* rows;
    int64_t rs;
    void* out;
    int64_t os;
};
hipError_t launch_combine_rows(const CombineRowsArgs& a, hipStream_t s);

struct CombineGradArgs {
    int T, k, d, dtype;
    const int32_t* inv;
    const float* w;
    const void* rows;             // nullptr iff dw is
    int64_t rs;
    const void* dout;
    int64_t dos;
    void* drows;                  // nullptr: skip
    int64_t drs;
    float* dw;                    // nullptr: skip
};
hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t s);

hipError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t R, int C, int64_t xs, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t R, int C, int dtype,
                                   void* out, int64_t os, hipStream_t s);

struct ProductArgs {
    int M, N, K, G;
    const void* a;                // bf16 [M][K] (stride as), or MXFP4 codes [M][K/2], or MXFP8 codes [M][K]
    const uint8_t* a_s;           // nullptr: bf16 rows
    bool a8;                      // MXFP8 rows
    int64_t as;
    const uint8_t* w;             // [G][N][K/2]
    const uint8_t* w_s;           // [G][N][K/32]
    const int32_t* offsets;       // [G+1] or nullptr (one group of all rows)
    void* out;                    // forward [M][N]; backward [M][K]
    int out_dtype;
    int64_t os;
};
// cus: compute units of the device; a: the rows, or (backward) dout bf16 [M][N]
hipError_t launch_product(const ProductArgs& p, int cus, hipStream_t s);
hipError_t launch_product_tiles(const ProductArgs& p, int cus, hipStream_t s);  // many rows a group
hipError_t launch_product8_tiles(const ProductArgs& p, int cus, hipStream_t s);
bool product8_dwords(const ProductArgs& p);      // whether MXFP8 rows' and the weight's scales can be read in dwords
hipError_t launch_product_grad(const ProductArgs& p, int cus, hipStream_t s);
hipError_t launch_product_grad_tiles(const ProductArgs& p, int cus, hipStream_t s);

}  // namespace moe

// Whether a product (or its gradient) takes the streaming kernels (1) or the tiles (0): the
// launches' own rule, device-free, for sizes that the product takes.  Exported so that the
// tests can say which kernel their shapes reach.  mx: 0 bf16 rows, 1 MXFP4, 2 MXFP8.
extern "C" int moe_internal_product_streams(int M, int N, int K, int G, int64_t stride, int mx, int backward,
                                            int cus);
// Of a product of MXFP8 rows in tiles: whether they are the short ones.
extern "C" int moe_internal_product8_short(int M, int N, int K, int G, int cus);
