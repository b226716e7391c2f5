/*
 * moe_ops.h - the expert layer's steps as operators of their own, for AMD
 * Instinct MI355X (gfx950): for callers that bring another router, another
 * activation, MXFP4 weights, or that train through the layer.  C ABI, in the same
 * library as moe_nvfp4.h and under its conventions (status codes, last error,
 * caller-owned device memory, work enqueued on `stream`, no host
 * synchronisation, no allocation; each call may be captured in a HIP graph).
 *
 *   dispatch   the T x k (token, slot) pairs sorted by local expert and the token
 *              rows gathered in that order, and its gradient
 *   combine    each token's expert rows weighted and summed, and its gradient
 *   MXFP4      quantizer and dequantizer, and the product of rows sorted by expert
 *              with each expert's MXFP4 weight, and its gradient
 *
 * A chain: dispatch -> [quantize] -> product -> activation -> product -> combine.
 *
 * Conventions beyond moe_nvfp4.h:
 *   - Row strides are in elements and at least the row's width; elements of a row
 *     are contiguous.  Rows of any stride and base address that keep their
 *     elements aligned are taken, except where a call asks for more.
 *   - Outputs must not overlap inputs or each other (INVALID_ARG).  Rows may take
 *     different columns of one buffer: strided tensors whose rows interleave are told
 *     apart by their columns modulo the greatest common divisor of their row strides.
 *   - Sums, products and dot products are fp32; each result is rounded once to its
 *     type.  No atomic decides an order: equal inputs give equal bits.
 *   - ARCH when the current device is not gfx950.
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_BF16 = 0,
    MOE_F16 = 1,
    MOE_F32 = 2,
    MOE_U8 = 3      /* dispatch only: rows of bytes (quantized codes or scales) */
} moe_dtype;

/* ------------------------------------------------------------------------- *
 * Dispatch and combine.
 *
 * Pair (t, j) of token t and slot j carries expert ids[t][j]; it is kept iff
 * 0 <= ids[t][j] - local_expert_offset < num_local_experts (an id outside the
 * model, e.g. -1 for a padded token or slot, is never kept).  The kept pairs are
 * sorted by (local expert, t, j); the same expert may stand in several slots of a
 * token.  P = their number, known on the device only.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t num_tokens;           /* T >= 0; T * top_k <= 2^27               */
    int32_t top_k;                /* k: 1..32                                */
    int32_t num_experts;          /* E: 1..1024                              */
    int32_t local_expert_offset;  /* o >= 0                                  */
    int32_t num_local_experts;    /* L >= 1, o + L <= E                      */
    int32_t width;                /* d: elements of a row, 1..65536          */
    int32_t dtype;                /* moe_dtype of the rows                   */
} moe_dispatch_problem;

/* Bytes of workspace moe_dispatch needs for `p` (0 for small batches).
 * Device-free. */
int moe_dispatch_workspace_size(const moe_dispatch_problem *p, size_t *bytes);

/* The plan and the gathered rows:
 *   ids     int32 [T][k]
 *   x       [T][d], row stride x_stride (NULL with rows == NULL: the plan alone)
 *   counts  int32 [L]      kept pairs per local expert
 *   offsets int32 [L+1]    exclusive scan of counts; offsets[L] = P
 *   perm    int32 [T*k]    first P entries: pair ids t*k+j in sorted order; the
 *                          rest is left as it was
 *   inv     int32 [T][k]   row of each pair, -1 if it is not kept
 *   rows    [T*k][d], row stride rows_stride: row r = x[perm[r] / k] for r < P,
 *           copied bit for bit; the rest is left as it was
 * counts, offsets, perm and inv may each be NULL to skip that output. */
int moe_dispatch(const moe_dispatch_problem *p, const int32_t *ids, const void *x, int64_t x_stride,
                 int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *inv, void *rows,
                 int64_t rows_stride, void *workspace, size_t workspace_bytes, void *stream);

/* Gradient of the gathered rows: dx[t] = sum over the kept slots, in slot order,
 * of drows[inv[t][j]] (0 for a token without one).  dtype bf16, f16 or f32.
 * Entries of inv outside [0, T*k) count as not kept, here and below. */
int moe_dispatch_backward(const moe_dispatch_problem *p, const int32_t *inv, const void *drows,
                          int64_t drows_stride, void *dx, int64_t dx_stride, void *stream);

/* out[t] = sum over the kept slots, in slot order, of weights[t][j] *
 * rows[inv[t][j]] (0 for a token without one; the weight of a slot that is not
 * kept is not looked at).  weights fp32 [T][k]; dtype bf16, f16 or f32. */
int moe_combine(const moe_dispatch_problem *p, const int32_t *inv, const float *weights, const void *rows,
                int64_t rows_stride, void *out, int64_t out_stride, void *stream);

/* Gradients of moe_combine from dout [T][d] (the kept entries of inv distinct, as
 * moe_dispatch leaves them: what a row that two pairs name holds is not specified):
 *   drows    [T*k][d]  drows[inv[t][j]] = weights[t][j] * dout[t]; other rows are
 *                      left as they were (NULL to skip)
 *   dweights fp32 [T][k] = dout[t] . rows[inv[t][j]], 0 where not kept (NULL to
 *                      skip; rows may then be NULL) */
int moe_combine_backward(const moe_dispatch_problem *p, const int32_t *inv, const float *weights,
                         const void *rows, int64_t rows_stride, const void *dout, int64_t dout_stride,
                         void *drows, int64_t drows_stride, float *dweights, void *stream);

/* ------------------------------------------------------------------------- *
 * MXFP4 (the Open Compute Project's microscaling format): E2M1 codes as in
 * NVFP4 (two per byte, the even element in the low nibble), one E8M0 scale byte s
 * per 32 consecutive elements of a row, value = code * 2^(s - 127); s = 255 makes
 * the block NaN.  gfx950's matrix cores multiply this format as it is.
 *
 * Quantizer: s = max(E - 2, 0) with E the biased fp32 exponent of the block's
 * largest magnitude (floor(log2 amax) - 2, clamped at 2^-127); code = E2M1 of
 * x / 2^(s - 127), round to nearest, ties to the even code, saturating at 6, the
 * sign of a zero kept; a block that holds an Inf or NaN gets s = 255, codes 0.
 * ------------------------------------------------------------------------- */

/* x [R][C] (bf16, f16 or f32; C a multiple of 32; R * C <= 2^40), row stride
 * x_stride -> codes u8 [R][C/2] (16-byte aligned), scales u8 [R][C/32], dense. */
int moe_mxfp4_quantize(const void *x, int32_t dtype, int64_t R, int32_t C, int64_t x_stride, uint8_t *codes,
                       uint8_t *scales, void *stream);

/* The values: out [R][C] (bf16, f16 or f32), row stride out_stride.  Exact in
 * bf16 and f32 up to overflow; rounded to nearest in f16 (overflow gives Inf). */
int moe_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t R, int32_t C, int32_t dtype,
                         void *out, int64_t out_stride, void *stream);

/* Rows sorted by group (expert) times each group's weight.  Group g owns rows
 * [offsets[g], offsets[g+1]) (device int32 [groups+1], e.g. moe_dispatch's;
 * clamped to [0, rows]; must not decrease); offsets NULL with groups == 1: all
 * rows.  Rows of no group are neither read nor written.
 *
 * Every scale byte counts as the format says, subnormal values too, with one bound:
 * W4A16 and the gradient hold weights in bf16, where a value of 2^128 or more (codes
 * from 4 on under s = 253, from 2 on under 254) is Inf. */
typedef struct {
    int32_t rows;      /* M: 0..2^27, rows of the buffers (an upper bound of the groups'    */
                       /* rows; M / G decides the kernel, so a near bound is the faster)    */
    int32_t n;         /* N: 1..65536, output features                                      */
    int32_t k;         /* K: a multiple of 32, 32..65536, the reduction                     */
    int32_t groups;    /* G: 1..1024                                                        */
} moe_product_problem;

/* out[r] = a[r] . w[g(r)]^T for the rows of every group.
 *   a        a_scales == NULL (W4A16): bf16 [M][K], row stride a_stride (a multiple
 *            of 8), 16-byte aligned;
 *            else (W4A4): MXFP4 codes u8 [M][K/2], 16-byte aligned, dense
 *            (a_stride is ignored), with a_scales u8 [M][K/32]
 *   w        MXFP4 codes u8 [G][N][K/2], 16-byte aligned; w_scales u8 [G][N][K/32]
 *   out      [M][N] of out_dtype (bf16, f16 or f32), row stride out_stride */
int moe_mxfp4_product(const moe_product_problem *p, const void *a, const uint8_t *a_scales, int64_t a_stride,
                      const uint8_t *w, const uint8_t *w_scales, const int32_t *offsets, void *out,
                      int32_t out_dtype, int64_t out_stride, void *stream);

/* Gradient of the rows (the weights are frozen; the W4A4 rows' rounding counts as
 * the identity): drows[r] = dout[r] . w[g(r)].
 *   dout   bf16 [M][N], row stride dout_stride
 *   drows  [M][K] of drows_dtype (bf16, f16 or f32), row stride drows_stride */
int moe_mxfp4_product_backward(const moe_product_problem *p, const void *dout, int64_t dout_stride,
                               const uint8_t *w, const uint8_t *w_scales, const int32_t *offsets, void *drows,
                               int32_t drows_dtype, int64_t drows_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_OPS_H */
