/*
 * moe_block.h - what stands round the expert layer's products, as operators of their
 * own, for AMD Instinct MI355X (gfx950).  C ABI, in the same library as moe_nvfp4.h and
 * moe_ops.h and under their conventions (status codes, last error, caller-owned device
 * memory, work enqueued on `stream`, no host synchronisation, no allocation, fixed orders
 * of sums, outputs that overlap nothing; each call may be captured in a HIP graph).
 *
 *   route     router logits to expert ids and weights, and the logits' gradient
 *   norm      a residual's addition and the root-mean-square norm, out in the rows' type
 *             and as MXFP8, and its gradients
 *   SwiGLU    the activation between the products, out in the rows' type and as MXFP8, its
 *             input kept as MXFP8 for the way back, and its gradient
 *   MXFP8     quantizer, dequantizer, and the product of MXFP8 rows with MXFP4 weights
 *             (W4A8)
 *
 * A chain: norm -> (logits) -> route -> moe_dispatch -> product -> SwiGLU -> product ->
 * moe_combine, and back.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------- *
 * Route.  Of a token's logits l [E] and an optional bias b [E]:
 *   score  s_e = softmax(l)_e or 1 / (1 + exp(-l_e))
 *   key    s_e + b_e, which the choice goes by (the weights do not see the bias)
 *   groups E / num_groups neighbouring experts each; with top_groups < num_groups only
 *          the experts of the top_groups groups with the highest sum of their group_keys
 *          highest keys (their only key, of a group of one) may be chosen
 *   ids    the top_k highest keys among them, highest first; equal keys: lower id first
 *   w_j    scale * s_{ids_j}, with `renormalize` divided by the sum of the chosen scores
 * An expert whose logit or bias is NaN or -Inf has no key and is never chosen (a logit of
 * NaN or -Inf has score 0).  A logit of +Inf counts as the largest finite fp32.  Where
 * fewer than top_k experts have keys the last ids are -1, their weights 0 (a group
 * without keys comes last; of groups with equal sums the lower one is first); chosen scores
 * that sum to 0 give weights of 0.
 *
 * The order is that of the exact keys: keys are compared in fp64, or by their logits
 * where no bias and no groups are given.  (moe_dispatch drops ids of -1, moe_combine does
 * not look at their weights.)
 * ------------------------------------------------------------------------- */
typedef enum { MOE_ROUTE_SOFTMAX = 0, MOE_ROUTE_SIGMOID = 1 } moe_route_scores;

typedef struct {
    int32_t num_tokens;     /* T >= 0; T * top_k <= 2^27                              */
    int32_t num_experts;    /* E: 1..1024                                             */
    int32_t top_k;          /* 1..32, at most top_groups * E / num_groups             */
    int32_t scores;         /* moe_route_scores                                       */
    int32_t num_groups;     /* 1..64, divides E                                       */
    int32_t top_groups;     /* 1..num_groups                                          */
    int32_t group_keys;     /* 1 or 2: keys of a group that its own is the sum of     */
    int32_t renormalize;    /* 0 or 1                                                 */
    int32_t dtype;          /* of the logits: bf16, f16 or f32                        */
    float scale;            /* finite                                                 */
} moe_route_problem;

/*   logits   [T][E], row stride logits_stride
 *   bias     fp32 [E], or NULL: none
 *   ids      int32 [T][k];  weights fp32 [T][k] */
int moe_route(const moe_route_problem *p, const void *logits, int64_t logits_stride, const float *bias, int32_t *ids,
              float *weights, void *stream);

/* Gradient of the logits from the weights', ids held fixed (the bias gets none):
 *   dlogits [T][E] of the logits' dtype, row stride dlogits_stride.
 * Entries of ids outside [0, E) count as not chosen; one that stands twice counts twice. */
int moe_route_backward(const moe_route_problem *p, const void *logits, int64_t logits_stride, const int32_t *ids,
                       const float *dweights, void *dlogits, int64_t dlogits_stride, void *stream);

/* ------------------------------------------------------------------------- *
 * Norm.  h = x + residual (rounded to the rows' type; h = x without a residual),
 *   rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight,
 * in fp32: a row whose sum of squares passes its range (from magnitudes of 2^64 / sqrt(d) on,
 * where all are alike: 2^58 at d = 4096) has rstd 0 and y 0; a mean square below 2^-25 eps leaves
 * no trace.  With eps 0 squares below 2^-126 lose bits, a row whose squares all vanish (magnitudes
 * below 2^-75) has rstd Inf, and of a row of zeros y is NaN.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t rows;           /* T: 0..2^27                                             */
    int32_t width;          /* d: 1..65536                                            */
    int32_t dtype;          /* of x, residual, h, y and their gradients               */
    int32_t weight_dtype;   /* bf16, f16 or f32                                       */
    float eps;              /* finite, >= 0                                           */
} moe_norm_problem;

/*   x, residual  [T][d], row strides (residual NULL: none)
 *   weight       [d]
 *   h            [T][d] (NULL to skip)
 *   y            [T][d] (NULL to skip)
 *   codes u8 [T][d] (16-byte aligned), scales u8 [T][d/32]: y as MXFP8, quantized from
 *                its fp32 value (both NULL to skip; d a multiple of 32 otherwise)
 *   rstd         fp32 [T] (NULL to skip) */
int moe_norm(const moe_norm_problem *p, const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
             const void *weight, void *h, int64_t h_stride, void *y, int64_t y_stride, uint8_t *codes, uint8_t *scales,
             float *rstd, void *stream);

/* Bytes of workspace moe_norm_backward needs for dweight.  Device-free. */
int moe_norm_workspace_size(const moe_norm_problem *p, size_t *bytes);

/* Gradients (the rounding of MXFP8 and of h counts as the identity).  With n = h * rstd:
 *   dx      [T][d] = rstd * (weight * dy - n * mean(weight * dy * n)) + dh: of x and of the
 *           residual alike (NULL to skip)
 *   dweight fp32 [d] = sum over the rows of dy * n (NULL to skip)
 *   dh      [T][d]: what else arrives at h (NULL: nothing)
 *   workspace: for dweight; calls that share one must not overlap */
int moe_norm_backward(const moe_norm_problem *p, const void *h, int64_t h_stride, const void *weight,
                      const float *rstd, const void *dy, int64_t dy_stride, const void *dh, int64_t dh_stride, void *dx,
                      int64_t dx_stride, float *dweight, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------- *
 * SwiGLU.  Rows u [M][2F] hold gate | up (the order of w13's outputs):
 *   a = gate / (1 + exp(-gate)) * up,
 * in fp32: from gates of about -88 downwards exp(-gate) passes its range, and a and du are 0 (their
 * values are below 2^-121 of |up|, and of |da up| and |da|).
 * offsets as the products' (device int32 [groups + 1]): rows from offsets[groups] on are
 * neither read nor written; NULL: all rows.
 * ------------------------------------------------------------------------- */
typedef struct {
    int32_t rows;           /* M: 0..2^27                                             */
    int32_t width;          /* F: 1..65536                                            */
    int32_t groups;         /* 1..1024                                                */
    int32_t dtype;          /* of u, a and their gradients: bf16, f16 or f32          */
} moe_swiglu_problem;

/*   u        [M][2F], row stride u_stride
 *   a        [M][F], row stride a_stride (NULL to skip)
 *   codes u8 [M][F] (16-byte aligned), scales u8 [M][F/32]: a as MXFP8, quantized from its
 *            fp32 value (both NULL to skip)
 *   kept u8 [M][2F] (16-byte aligned), kept_scales u8 [M][2F/32]: u as MXFP8, for the way
 *            back in half the bytes (both NULL to skip)
 * F is a multiple of 32 where MXFP8 is written. */
int moe_swiglu(const moe_swiglu_problem *p, const void *u, int64_t u_stride, const int32_t *offsets, void *a,
               int64_t a_stride, uint8_t *codes, uint8_t *scales, uint8_t *kept, uint8_t *kept_scales, void *stream);

/* du [M][2F] = (da * up * s * (1 + gate * (1 - s)) | da * gate * s), s = 1 / (1 + exp(-gate)).
 *   u         kept_scales == NULL: rows [M][2F] of dtype, row stride u_stride;
 *             else: MXFP8 codes u8 [M][2F], 16-byte aligned, dense (u_stride is ignored),
 *             with kept_scales u8 [M][2F/32]; F a multiple of 32
 *   da        [M][F], row stride da_stride;  du [M][2F], row stride du_stride */
int moe_swiglu_backward(const moe_swiglu_problem *p, const void *u, int64_t u_stride, const uint8_t *kept_scales,
                        const int32_t *offsets, const void *da, int64_t da_stride, void *du, int64_t du_stride,
                        void *stream);

/* ------------------------------------------------------------------------- *
 * MXFP8 (the Open Compute Project's microscaling format): E4M3 codes, one a byte, one
 * E8M0 scale byte s per 32 consecutive elements of a row, value = code * 2^(s - 127); s =
 * 255 makes the block NaN.
 *
 * Quantizer: s = max(E - 8, 0) with E the biased fp32 exponent of the block's largest
 * magnitude (floor(log2 amax) - 8, clamped at 2^-127); code = E4M3 of x / 2^(s - 127),
 * round to nearest, ties to even, saturating at 448, the sign of a zero kept; a block
 * that holds an Inf or NaN gets s = 255, codes 0.
 * ------------------------------------------------------------------------- */

/* x [R][C] (bf16, f16 or f32; C a multiple of 32; R * C <= 2^40), row stride x_stride ->
 * codes u8 [R][C] (16-byte aligned), scales u8 [R][C/32], dense. */
int moe_mxfp8_quantize(const void *x, int32_t dtype, int64_t R, int32_t C, int64_t x_stride, uint8_t *codes,
                       uint8_t *scales, void *stream);

/* The values: out [R][C] (bf16, f16 or f32), row stride out_stride.  Exact in f32, and in bf16
 * under scale bytes from 3 on, up to overflow; rounded to nearest in f16 (overflow gives Inf) and
 * under the three lowest scale bytes in bf16, whose smallest value 2^-133 is above theirs. */
int moe_mxfp8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t R, int32_t C, int32_t dtype, void *out,
                         int64_t out_stride, void *stream);

/* out[r] = a[r] . w[g(r)]^T for the rows of every group: moe_mxfp4_product with MXFP8 rows.
 * (Its gradient is moe_mxfp4_product_backward: the rows' rounding counts as the identity.)
 *   a   MXFP8 codes u8 [M][K], 16-byte aligned, dense, with a_scales u8 [M][K/32]
 * The matrix cores add the products of eight neighbouring k after aligning them to the
 * largest, and drop what lies 2^-13 of it and lower; the sums of eights are fp32. */
int moe_mxfp8_product(const moe_product_problem *p, const uint8_t *a, const uint8_t *a_scales, const uint8_t *w,
                      const uint8_t *w_scales, const int32_t *offsets, void *out, int32_t out_dtype,
                      int64_t out_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
