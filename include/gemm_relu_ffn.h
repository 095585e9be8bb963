/*
 * Operators of a transformer's feed-forward half layer on AMD Instinct MI355X
 * (gfx950): layer norm, the gated projections and the 8-bit integer product,
 * with the backward passes and the row quantisation they need.  Part of
 * libgemm_relu.so; the type and status codes are those of gemm_relu.h.
 *
 * Common to every call:
 *   - Tensors are device pointers to row-major matrices.  A *_stride argument
 *     counts elements from one row to the next (>= the row's length); matrices
 *     without one are dense.  Pointers need the alignment of their element.
 *   - Sizes are >= 0 and <= INT32_MAX.  A call whose outputs have no elements
 *     returns GEMM_RELU_OK without touching the device.
 *   - Sums, means and statistics are fp32 (int32 where stated), and so are the
 *     operations behind them; results are then rounded to their type, to nearest
 *     even.  Results are the same bits on every run: nothing is summed in an order
 *     that depends on timing.
 *   - The call allocates nothing and is asynchronous on `stream` (a hipStream_t
 *     or NULL); it may be captured into a graph.  The library keeps no pointer.
 *     GEMM_RELU_SYNC=1 in the environment makes it synchronise and report.
 *   - A workspace is caller's device memory, 256-byte aligned, of at least the
 *     bytes the matching *_workspace function returns.  Its contents need no
 *     preparation.  Calls that may overlap need one each.
 *   - Errors: GEMM_RELU_EINVAL for a bad size, stride, code or alignment, a NULL
 *     pointer to a tensor with elements, a workspace that is too small, or an
 *     output that overlaps an input or another output (checked before any HIP
 *     call); GEMM_RELU_EUNSUPPORTED where the device is no gfx950, a stated limit
 *     is passed, or a product would take more than 2^22 workgroups (tiles of the
 *     configuration that its *_plan function names); GEMM_RELU_EHIP when a HIP call
 *     fails.  Both of the former launch nothing.
 */
#ifndef GEMM_RELU_FFN_H
#define GEMM_RELU_FFN_H

#include <stdint.h>

#include "gemm_relu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the gated projections. */
#define GEMM_RELU_ACT_SILU      0 /* g / (1 + e^-g) */
#define GEMM_RELU_ACT_GELU      1 /* g Phi(g), Phi the normal distribution function */
#define GEMM_RELU_ACT_GELU_TANH 2 /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
#define GEMM_RELU_ACT_RELU      3 /* max(g, 0) */

/*
 * Layer norm of each row of x (rows x cols):
 *   mean = sum_j x_j / cols,  rstd = (sum_j (x_j - mean)^2 / cols + eps)^(-1/2),
 *   y_j = (x_j - mean) rstd weight_j + bias_j.
 * dtype (x, y): F16, BF16 or F32.  wdtype (weight, bias): dtype or F32.  bias
 * may be NULL (zero).  mean and rstd (rows floats each) are written unless NULL.
 * cols >= 1; eps >= 0.  A row with an infinity or NaN gives a row of NaN, and
 * so does one whose sum passes fp32; one whose squared distances from the mean pass
 * it (distances above 1.8e19) has rstd 0.
 */
int gemm_relu_layer_norm(const void* x, int64_t x_stride, const void* weight, const void* bias,
                         void* y, float* mean, float* rstd, int64_t rows, int64_t cols, int dtype,
                         int wdtype, float eps, void* stream);

/*
 * Its backward pass.  With xhat = (x - mean) rstd and c_j = dy_j weight_j:
 *   dx_j = rstd (c_j - sum_k c_k / cols - xhat_j sum_k c_k xhat_k / cols),
 *   dweight_j = sum over rows of dy_j xhat_j,  dbias_j = sum over rows of dy_j.
 * dx has dtype, dweight and dbias (cols elements each) have wdtype; dbias may
 * be NULL.  mean and rstd are the forward call's.  rows == 0 writes zeros to
 * dweight and dbias.
 */
int64_t gemm_relu_layer_norm_backward_workspace(int64_t rows, int64_t cols);
int gemm_relu_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x,
                                  int64_t x_stride, const void* weight, const float* mean,
                                  const float* rstd, void* dx, void* dweight, void* dbias,
                                  int64_t rows, int64_t cols, int dtype, int wdtype,
                                  void* workspace, uint64_t workspace_bytes, void* stream);

/*
 * Gated projections: with the weight's first `hidden` rows Wg and its last
 * `hidden` rows Wu (weight is 2 hidden x cols),
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) u      (rows x hidden).
 * dtype (x, weight, h): F16 or BF16.  gu, unless NULL, receives the fp32 sums
 * for the backward pass: rows x 2 hidden, g then u in each row.  2 hidden and
 * every stride <= INT32_MAX; cols <= INT32_MAX - 127, else
 * GEMM_RELU_EUNSUPPORTED.  cols == 0 gives zeros.
 */
int gemm_relu_gated(const void* x, int64_t x_stride, const void* weight, int64_t weight_stride,
                    void* h, float* gu, int64_t rows, int64_t hidden, int64_t cols, int dtype,
                    int act, void* stream);

/* Name of the kernel configuration gemm_relu_gated would launch for dense rows
 * ("a+b" where the last rows take a second launch; "none" for an empty call,
 * "unsupported" above a stated limit, NULL for invalid sizes or codes).  Rows more
 * than 2^22 elements apart can take another.  The text stays valid.  Host-only. */
const char* gemm_relu_gated_plan(int64_t rows, int64_t hidden, int64_t cols, int dtype);

/*
 * Their backward pass, from dh (rows x hidden) and the forward call's gu:
 *   dg = dh u act'(g),  du = dh act(g),  dx = dg Wg + du Wu,
 *   dweight = [dg^T x; du^T x]                  (2 hidden x cols).
 * dg and du are rounded to dtype before the two products, whose matrix
 * instructions take 16-bit inputs (F16 values below its normal range to a multiple
 * of 2^-24).  Where a finite dg or du would become an F16 infinity, its row of dx
 * and its row of dweight are summed in fp32 without that rounding.  max(g, 0) has slope 0 at 0.  rows and 2 hidden
 * <= 2^30, else GEMM_RELU_EUNSUPPORTED (from the workspace function too).
 */
int64_t gemm_relu_gated_backward_workspace(int64_t rows, int64_t hidden, int64_t cols);
int gemm_relu_gated_backward(const void* dh, int64_t dh_stride, const float* gu, const void* x,
                             int64_t x_stride, const void* weight, int64_t weight_stride,
                             void* dx, void* dweight, int64_t rows, int64_t hidden, int64_t cols,
                             int dtype, int act, void* workspace, uint64_t workspace_bytes,
                             void* stream);

/* Configuration names of its two products, "dx,dweight" (as above; other ones for rows
 * of x or weight more than 2^24 elements apart). */
const char* gemm_relu_gated_backward_plan(int64_t rows, int64_t hidden, int64_t cols, int dtype);

/*
 * Quantisation of each row of x (rows x cols; F16, BF16 or F32) to 8 bits:
 *   scale = max_k |x_k| / 127,  q_k = 127 x_k / max_k |x_k| rounded to the
 * nearest integer, ties to even (exactly so for 16-bit x).  q is rows x cols
 * int8, scale rows floats.  A row of zeros (or of no elements) has scale 0 and
 * q 0; a row with an infinity or NaN has scale NaN and q 0, so that products
 * with it are NaN.
 */
int gemm_relu_quantize_rows(const void* x, int64_t x_stride, void* q, float* scale, int64_t rows,
                            int64_t cols, int dtype, void* stream);

/*
 * 8-bit integer product: y_ij = (sum_k x_ik w_jk) x_scale_i w_scale_j for int8
 * x (rows x k) and w (n x k, one row per output channel), the sum exact in
 * int32, then rounded to fp32, as are its products with x_scale and with w_scale
 * (fp32 results so carry three roundings).  y is rows x n of out_dtype (F16, BF16 or F32).  k <= 131071 (where no
 * sum can overflow), else GEMM_RELU_EUNSUPPORTED.
 */
int gemm_relu_i8(const void* x, int64_t x_stride, const float* x_scale, const void* w,
                 int64_t w_stride, const float* w_scale, void* y, int64_t rows, int64_t n,
                 int64_t k, int out_dtype, void* stream);

/* Configuration name gemm_relu_i8 would launch (as gemm_relu_gated_plan). */
const char* gemm_relu_i8_plan(int64_t rows, int64_t n, int64_t k, int out_dtype);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RELU_FFN_H */
