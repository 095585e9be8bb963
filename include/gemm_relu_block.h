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
 * a multiple of 2^-23.  max(z, 0) has slope 0 at 0.  rows and n <= 2^30, else
 * GEMM_RELU_EUNSUPPORTED (from the workspace function too).
 */
int64_t gemm_relu_act_backward_workspace(int64_t rows, int64_t n, int64_t k);
int gemm_relu_act_backward(const void* dy, int64_t dy_stride, const float* z, const void* x,
                           int64_t x_stride, const void* weight, int64_t weight_stride, void* dx,
                           void* dweight, void* dbias, int64_t rows, int64_t n, int64_t k, int dtype,
                           int bias_dtype, int act, void* workspace, uint64_t workspace_bytes,
                           void* stream);

/* Configuration names of its two products, "dx,dweight". */
const char* gemm_relu_act_backward_plan(int64_t rows, int64_t n, int64_t k, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RELU_BLOCK_H */
