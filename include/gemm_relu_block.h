/*
 * Operators around a transformer's feed-forward half layer on AMD Instinct MI355X
 * (gfx950): the product with bias, activation and residual, the step from one block
 * to the next (residual sum and norms), both with their backward passes, and the
 * orthogonalisation of a weight's update.  Part of libgemm_relu.so.
 *
 * What gemm_relu_ffn.h says of every call holds here too: device pointers to
 * row-major matrices, strides in elements, fp32 sums with one rounding to the result's
 * type, the same bits on every run, no allocation, asynchronous on `stream`, workspaces,
 * error codes.  Sizes are >= 0 and <= INT32_MAX.
 */
#ifndef GEMM_RELU_BLOCK_H
#define GEMM_RELU_BLOCK_H

#include <stdint.h>

#include "gemm_relu.h"
#include "gemm_relu_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* No activation, beside the GEMM_RELU_ACT_* of gemm_relu_ffn.h. */
#define GEMM_RELU_ACT_NONE 4

/*
 * Product with bias, activation and residual:
 *   z = x weight^T + bias,  y = act(z) + residual        (rows x n)
 * for x (rows x k) and weight (n x k).  dtype (x, weight, residual, y): F16 or BF16.
 * bias (n; bias_dtype: dtype or F32) and residual may be NULL.  z, unless NULL, receives
 * the fp32 sums with the bias, which the backward pass of an activation takes.  k == 0
 * gives act(bias) + residual.  Every stride <= INT32_MAX; k <= INT32_MAX - 127, else
 * GEMM_RELU_EUNSUPPORTED.
 */
int gemm_relu_act(const void* x, int64_t x_stride, const void* weight, int64_t weight_stride,
                  const void* bias, const void* residual, int64_t residual_stride, void* y, float* z,
                  int64_t rows, int64_t n, int64_t k, int dtype, int bias_dtype, int act, void* stream);

/* Configuration name, as gemm_relu_gated_plan's. */
const char* gemm_relu_act_plan(int64_t rows, int64_t n, int64_t k, int dtype);

/*
 * Its backward pass, from dy (rows x n) and the forward call's z (NULL with
 * GEMM_RELU_ACT_NONE, which needs none):
 *   dz = dy act'(z),  dx = dz weight,  dweight = dz^T x,  dbias = sum over rows of dz;
 * the residual's gradient is dy itself.  dx and dweight have dtype; dbias (n, of
 * bias_dtype) may be NULL.  dz is rounded to dtype before the products (the sum over
 * rows takes it as it is); with F16 and an activation but max(z, 0), whose slopes pass
 * 1, half of it is, so that no finite dy gives an infinite dz: below 2^-13 it is then
 * a multiple of 2^-23.  max(z, 0) has slope 0 at 0.  The lower tail of gelu's distribution
 * function, here and in gemm_relu_act, is within 6e-6 of itself for |z| < 8.  rows and n <=
 * 2^30, else GEMM_RELU_EUNSUPPORTED (from the workspace function too), and so are
 * matrices dz of 2^23 or more tiles of 64 x 64 (from the call).
 */
int64_t gemm_relu_act_backward_workspace(int64_t rows, int64_t n, int64_t k);
int gemm_relu_act_backward(const void* dy, int64_t dy_stride, const float* z, const void* x,
                           int64_t x_stride, const void* weight, int64_t weight_stride, void* dx,
                           void* dweight, void* dbias, int64_t rows, int64_t n, int64_t k, int dtype,
                           int bias_dtype, int act, void* workspace, uint64_t workspace_bytes,
                           void* stream);

/* Configuration names of its two products, "dx,dweight". */
const char* gemm_relu_act_backward_plan(int64_t rows, int64_t n, int64_t k, int dtype);

/* Norms of gemm_relu_add_norm: v / sqrt(mean v^2 + eps), and gemm_relu_layer_norm's. */
#define GEMM_RELU_NORM_RMS   0
#define GEMM_RELU_NORM_LAYER 1

/*
 * From one block to the next: the block's output x, normed first if post_weight is
 * given, gated and scaled, is added to the residual stream, whose sum the next block's
 * norm takes (rows past fp32's range: as gemm_relu_layer_norm; with eps 0, squares of values
 * under 2^-63 lose digits, and a row of values under 2^-75 has an infinite 1 / deviation).  For
 * each row of x and residual (rows x cols),
 *   t = norm(x) post_weight, or x without one,
 *   s = residual + scale gate t,
 *   y = norm(s) weight + bias.
 * gate: NULL (1), one row for all (gate_stride 0; cols elements of wdtype), or a matrix
 * like x (gate_stride >= cols; of dtype).  weight NULL: no y (NULL too, as bias).  bias
 * and post_weight may be NULL.  dtype (x, residual, s, y): F16, BF16 or F32; wdtype
 * (weight, bias, post_weight): dtype or F32.  y is made of the fp32 s, not of the rounded
 * one.  stats, unless NULL, receives 4 floats a row for the backward pass.  cols >= 1;
 * eps >= 0; scale finite.
 */
int gemm_relu_add_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                       const void* gate, int64_t gate_stride, const void* post_weight,
                       const void* weight, const void* bias, void* s, void* y, float* stats,
                       int64_t rows, int64_t cols, int dtype, int wdtype, int norm, float scale,
                       float eps, void* stream);

/*
 * Its backward pass, from dy (NULL without a weight), the gradient ds that reaches s from
 * elsewhere (NULL: none) and the forward call's stats:
 *   dresidual = ds + (the norm's gradient of dy weight at s),  dt = scale gate dresidual,
 *   dgate = scale t dresidual (summed over rows for a gate of one row),
 *   dpost_weight = sum over rows of dt (norm(x)),  dx = the norm's gradient of
 *   dt post_weight at x, or dt,  dweight = sum over rows of dy (norm(s)),  dbias = sum over
 *   rows of dy.
 * s is computed again from x and residual, so nothing is lost in its rounding.  Every
 * output may be NULL: not wanted (dx is dresidual without gate and post_weight and with
 * scale 1; dresidual is ds without a weight).  dx, dresidual and a matrix's dgate have
 * dtype, the others wdtype.  rows == 0 writes zeros to the sums over rows.
 */
int64_t gemm_relu_add_norm_backward_workspace(int64_t rows, int64_t cols);
int gemm_relu_add_norm_backward(const void* dy, int64_t dy_stride, const void* ds, int64_t ds_stride,
                                const void* x, int64_t x_stride, const void* residual,
                                int64_t residual_stride, const void* gate, int64_t gate_stride,
                                const void* post_weight, const void* weight, const float* stats,
                                void* dx, void* dresidual, void* dgate, void* dpost_weight,
                                void* dweight, void* dbias, int64_t rows, int64_t cols, int dtype,
                                int wdtype, int norm, float scale, void* workspace,
                                uint64_t workspace_bytes, void* stream);

/*
 * Orthogonalisation of matrices by Newton-Schulz steps: each of the batch's matrices g
 * (rows x cols, batch_stride elements apart, 0 to 2^40) becomes
 *   X = g / (|g| + eps), |g| the square root of the sum of squares,
 *   X <- a X + (b A + c A^2) X,  A = X X^T,   once per step with its a, b, c,
 * (with A = X^T X on the right where rows > cols: the same matrix).  The singular vectors
 * stay, the singular values tend to 1.  coefficients: host memory, steps times a, b, c,
 * read before the call returns; steps <= 64.  dtype (g): F16, BF16 or F32.  out is dense
 * bfloat16 (batch x rows x cols).  X is kept in two float16 (22 bits; fp32 where a call of a
 * short side is one launch, or one a step), and b A + c A^2 multiplies both; A is made of
 * the larger, and A's and b A + c A^2's values off their diagonals are rounded to float16 as
 * operands.  What a result is off before it is rounded, as a share of its norm and whatever
 * the singular values: with (3.4445, -4.7750, 2.0315) 3e-3 for up to 6 steps where the shorter
 * side is at least 16 (5e-4 is usual) and 1e-2 for up to 5 below that; with (1.5, -0.5, 0) and
 * (1.875, -1.25, 0.375), which converge, 1.5e-3 for up to 12 steps.  The former do not
 * converge: their singular values keep moving, by factors of up to 1.6 further apart a step,
 * which takes 3e-3 to 1.2e-2 after 10 steps.  Coefficients of larger slopes grow their
 * roundings accordingly.  A singular value below 2^-22 of the norm is lost in X, as one below
 * 2^-24 is in fp32, and many steps of a large a bring what is there instead up to 1.
 * Values of X and of b A + c A^2 past 2^8 in magnitude, and of A past 2^6, are past
 * float16's range here and give infinities and NaN; coefficients that keep the singular
 * values below 2 stay far from that.  A matrix of zeros gives zeros (with eps == 0 NaN, 0 /
 * 0); a NaN in g, or with at least one step an infinity, gives NaN all over its matrix.  The
 * shorter side <= 2^16, the longer <= 2^22, rows x cols <= 2^34, batch <= 65535, else
 * GEMM_RELU_EUNSUPPORTED.
 */
int64_t gemm_relu_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols);
int gemm_relu_orthogonalize(const void* g, int64_t g_stride, int64_t batch_stride, void* out,
                            int64_t batch, int64_t rows, int64_t cols, int dtype,
                            const float* coefficients, int steps, float eps, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Configuration names of a step's products, "A,B,X" ("t/d" where a symmetric one's tiles on
 * the diagonal take another configuration d, "t*n" where A's K is cut into n parts; "small"
 * where one launch does all steps, "long" where one does a step, "none", "unsupported" and
 * NULL as for the others).  The text stays valid.  Host-only. */
const char* gemm_relu_orthogonalize_plan(int64_t batch, int64_t rows, int64_t cols);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RELU_BLOCK_H */
