// C-ABI of the feed-forward operators (include/gemm_relu_ffn.h): argument checks,
// configuration choice, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_common.hpp"
#include "ffn.hpp"
#include "gemm_relu_ffn.h"
#include "linear_plan.hpp"

using namespace gemm_relu_hip;

namespace {

// The plan of the gated projections' gradient, whose element-wise pass notes values past float16.
GradPlan plan_gated_grad(int64_t rows, int64_t hidden, int64_t cols, int64_t x_stride, int64_t weight_stride)
{
    return plan_grad(rows, 2 * hidden, cols, x_stride, weight_stride,
                     uint64_t(ceil_div(rows, 64) * ceil_div(hidden, 64)) * 3 * sizeof(GradMask));
}

}  // namespace

// ------------------------------------------------------------- layer norm
extern "C" int gemm_relu_layer_norm(const void* x, int64_t x_stride, const void* weight, const void* bias,
                                    void* y, float* mean, float* rstd, int64_t rows, int64_t cols, int dtype,
                                    int wdtype, float eps, void* stream)
{
    if (!size_ok(rows) || !size_ok(cols) || !is_float(dtype) || (wdtype != dtype && wdtype != GEMM_RELU_F32) ||
        !(eps >= 0.0f) || (rows > 0 && cols < 1))
        return GEMM_RELU_EINVAL;
    if (rows == 0) return GEMM_RELU_OK;
    const int e = elem_bytes(dtype), we = elem_bytes(wdtype);
    const Mat m[] = {dense(y, rows, cols, e), dense(mean, mean ? rows : 0, 1, 4), dense(rstd, rstd ? rows : 0, 1, 4),
                     {x, rows, cols, x_stride, e}, dense(weight, 1, cols, we), dense(bias, bias ? 1 : 0, cols, we)};
    if (!mats_ok(m, 3)) return GEMM_RELU_EINVAL;
    if (const int dev = check_device()) return dev;
    NormArgs a{};
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.x_stride = x_stride;
    a.rows = int(rows);
    a.cols = int(cols);
    a.eps = eps;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return finish(launch_layer_norm(a, dtype, wdtype, st), st);
}

extern "C" int64_t gemm_relu_layer_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (!size_ok(rows) || !size_ok(cols)) return GEMM_RELU_EINVAL;
    // of the type that leaves more strips
    return int64_t(std::max(layer_norm_strips(rows, cols, 2), layer_norm_strips(rows, cols, 4))) * 2 * cols * 4;
}

extern "C" int gemm_relu_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                                             const void* weight, const float* mean, const float* rstd, void* dx,
                                             void* dweight, void* dbias, int64_t rows, int64_t cols, int dtype,
                                             int wdtype, void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (!size_ok(rows) || !size_ok(cols) || !is_float(dtype) || (wdtype != dtype && wdtype != GEMM_RELU_F32) ||
        (rows > 0 && cols < 1))
        return GEMM_RELU_EINVAL;
    if (cols == 0) return GEMM_RELU_OK;
    const uint64_t need = uint64_t(gemm_relu_layer_norm_backward_workspace(rows, cols));
    const int e = elem_bytes(dtype), we = elem_bytes(wdtype);
    const Mat m[] = {dense(dx, rows, cols, e), dense(dweight, 1, cols, we), dense(dbias, dbias ? 1 : 0, cols, we),
                     bytes_of(workspace, need), {dy, rows, cols, dy_stride, e}, {x, rows, cols, x_stride, e},
                     dense(weight, 1, cols, we), dense(mean, rows, 1, 4), dense(rstd, rows, 1, 4)};
    if (!mats_ok(m, 4) || !workspace_ok(workspace, workspace_bytes, need)) return GEMM_RELU_EINVAL;
    if (const int dev = check_device()) return dev;
    NormArgs a{};
    a.x = x;
    a.w = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dx = dx;
    a.dw = dweight;
    a.db = dbias;
    a.partial = static_cast<float*>(workspace);
    a.x_stride = x_stride;
    a.dy_stride = dy_stride;
    a.rows = int(rows);
    a.cols = int(cols);
    hipStream_t st = static_cast<hipStream_t>(stream);
    return finish(launch_layer_norm_backward(a, dtype, wdtype, st), st);
}

// --------------------------------------------------------- gated projections
static bool gated_sizes_ok(int64_t rows, int64_t hidden, int64_t cols, int dtype)
{
    return size_ok(rows) && size_ok(hidden) && 2 * hidden <= kLim && size_ok(cols) && is_16bit(dtype);
}

// both projections' columns, dense rows unless told otherwise
static Linear gated_linear(int64_t rows, int64_t hidden, int64_t cols, int64_t lda, int64_t ldb)
{
    return Linear{rows, 2 * hidden, cols, lda, ldb, true};
}

extern "C" int gemm_relu_gated(const void* x, int64_t x_stride, const void* weight, int64_t weight_stride, void* h,
                               float* gu, int64_t rows, int64_t hidden, int64_t cols, int dtype, int act, void* stream)
{
    if (!gated_sizes_ok(rows, hidden, cols, dtype) || act < GEMM_RELU_ACT_SILU || act > GEMM_RELU_ACT_RELU)
        return GEMM_RELU_EINVAL;
    if (rows == 0 || hidden == 0) return GEMM_RELU_OK;
    const Mat m[] = {dense(h, rows, hidden, 2), dense(gu, gu ? rows : 0, 2 * hidden, 4),
                     {x, rows, cols, x_stride, 2}, {weight, 2 * hidden, cols, weight_stride, 2}};
    if (!mats_ok(m, 2)) return GEMM_RELU_EINVAL;
    const RowsPlan r = plan_rows(gated_linear(rows, hidden, cols, x_stride, weight_stride));
    if (cols > kMaxK || r.p.grid() > kMaxGrid) return GEMM_RELU_EUNSUPPORTED;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    auto go = [&](const LinearPlan& p, const Linear& l, int64_t first) {
        KernelArgs a = linear_args(p, l, static_cast<const char*>(x) + 2 * first * x_stride, weight,
                                   static_cast<char*>(h) + 2 * first * hidden);
        a.hidden = int(hidden);
        a.act = act;
        a.GU = gu ? gu + first * 2 * hidden : nullptr;
        return launcher_gated(dtype, p.cfg)(a, int(p.grid()), st);
    };
    hipError_t e = go(r.p, r.top, 0);
    if (e == hipSuccess && r.rest.M > 0) e = go(r.q, r.rest, r.top.M);
    return finish(e, st);
}

extern "C" const char* gemm_relu_gated_plan(int64_t rows, int64_t hidden, int64_t cols, int dtype)
{
    if (!gated_sizes_ok(rows, hidden, cols, dtype)) return nullptr;
    if (rows == 0 || hidden == 0) return "none";
    if (cols > kMaxK) return "unsupported";
    return rows_plan_name(plan_rows(gated_linear(rows, hidden, cols, cols, cols)));
}

extern "C" int64_t gemm_relu_gated_backward_workspace(int64_t rows, int64_t hidden, int64_t cols)
{
    if (!gated_sizes_ok(rows, hidden, cols, GEMM_RELU_F16)) return GEMM_RELU_EINVAL;
    if (cols == 0) return 0;
    if (rows > kMaxGradRows || 2 * hidden > kMaxGradRows) return GEMM_RELU_EUNSUPPORTED;
    return int64_t(plan_gated_grad(rows, hidden, cols, cols, cols).bytes);
}

extern "C" int gemm_relu_gated_backward(const void* dh, int64_t dh_stride, const float* gu, const void* x,
                                        int64_t x_stride, const void* weight, int64_t weight_stride, void* dx,
                                        void* dweight, int64_t rows, int64_t hidden, int64_t cols, int dtype,
                                        int act, void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (!gated_sizes_ok(rows, hidden, cols, dtype) || act < GEMM_RELU_ACT_SILU || act > GEMM_RELU_ACT_RELU)
        return GEMM_RELU_EINVAL;
    if (cols == 0 || (rows == 0 && hidden == 0)) return GEMM_RELU_OK;
    if (rows > kMaxGradRows || 2 * hidden > kMaxGradRows) return GEMM_RELU_EUNSUPPORTED;
    const GradPlan p = plan_gated_grad(rows, hidden, cols, x_stride, weight_stride);
    const Mat m[] = {dense(dx, rows, cols, 2), dense(dweight, 2 * hidden, cols, 2), bytes_of(workspace, p.bytes),
                     {dh, rows, hidden, dh_stride, 2}, dense(gu, rows, 2 * hidden, 4), {x, rows, cols, x_stride, 2},
                     {weight, 2 * hidden, cols, weight_stride, 2}};
    if (!mats_ok(m, 3) || !workspace_ok(workspace, workspace_bytes, p.bytes)) return GEMM_RELU_EINVAL;
    if (p.x.grid() + p.w.grid() > kMaxGrid || ceil_div(hidden, 64) * ceil_div(rows, 64) * kGradThreads >= (int64_t(1) << 32))
        return GEMM_RELU_EUNSUPPORTED;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    unsigned* flags = reinterpret_cast<unsigned*>(ws + p.flags);
    hipError_t e = hipSuccess;
    GatedGradArgs g{};
    const bool grad = rows > 0 && hidden > 0;
    if (grad) {
        g.gu = gu;
        g.dh = dh;
        g.dgu = ws;
        g.dgu_t = ws + p.dz_t;
        g.dh_stride = dh_stride;
        g.ld = int(p.lx.lda);
        g.ld_t = int(p.lw.lda);
        g.rows = int(rows);
        g.hidden = int(hidden);
        g.act = act;
        g.flags = flags;
        g.nflags = p.nflags();
        g.over = reinterpret_cast<GradMask*>(ws + p.more);
        g.x = x;
        g.w = weight;
        g.dx = dx;
        g.dw = dweight;
        g.x_stride = x_stride;
        g.w_stride = weight_stride;
        g.cols = int(cols);
        e = launch_gated_grad(g, dtype, st);
    }
    KernelArgs gx = linear_args(p.x, p.lx, ws, weight, dx), gw = linear_args(p.w, p.lw, ws + p.dz_t, x, dweight);
    gx.flags = flags;
    gx.ws = reinterpret_cast<float*>(ws + p.sums_x);
    gw.flags = flags + (p.x.splits > 1 ? p.x.tiles() : 0);
    gw.ws = reinterpret_cast<float*>(ws + p.sums_w);
    const int nx = rows > 0 ? int(p.x.grid()) : 0, nw = hidden > 0 ? int(p.w.grid()) : 0;
    if (e == hipSuccess) {
        // the product whose tiles take longest first
        const bool x_first = p.lx.K * p.w.splits >= p.lw.K * p.x.splits;
        e = launcher_cast_pair(dtype, p.x.cfg)(x_first ? LinearPair{gx, gw, nx} : LinearPair{gw, gx, nw}, nx + nw, st);
    }
    if (e == hipSuccess && grad && dtype == GEMM_RELU_F16) e = launch_gated_repair(g, st);
    return finish(e, st);
}

extern "C" const char* gemm_relu_gated_backward_plan(int64_t rows, int64_t hidden, int64_t cols, int dtype)
{
    if (!gated_sizes_ok(rows, hidden, cols, dtype)) return nullptr;
    if (cols == 0 || (rows == 0 && hidden == 0)) return "none";
    const GradPlan p = plan_gated_grad(rows, hidden, cols, cols, cols);
    static const PairNames names(',');
    return names.text[p.x.cfg][p.w.cfg];
}

// ------------------------------------------------------- 8-bit integers
extern "C" int gemm_relu_quantize_rows(const void* x, int64_t x_stride, void* q, float* scale, int64_t rows,
                                       int64_t cols, int dtype, void* stream)
{
    if (!size_ok(rows) || !size_ok(cols) || !is_float(dtype)) return GEMM_RELU_EINVAL;
    if (rows == 0) return GEMM_RELU_OK;
    const Mat m[] = {dense(q, rows, cols, 1), dense(scale, rows, 1, 4), {x, rows, cols, x_stride, elem_bytes(dtype)}};
    if (!mats_ok(m, 2)) return GEMM_RELU_EINVAL;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return finish(launch_quantize_rows(x, x_stride, static_cast<signed char*>(q), scale, int(rows), int(cols), dtype, st),
                  st);
}

constexpr int64_t kMaxK8 = 131071;      // 128 * 128 * k < 2^31

extern "C" int gemm_relu_i8(const void* x, int64_t x_stride, const float* x_scale, const void* w, int64_t w_stride,
                            const float* w_scale, void* y, int64_t rows, int64_t n, int64_t k, int out_dtype,
                            void* stream)
{
    if (!size_ok(rows) || !size_ok(n) || !size_ok(k) || !is_float(out_dtype)) return GEMM_RELU_EINVAL;
    if (rows == 0 || n == 0) return GEMM_RELU_OK;
    const Mat m[] = {dense(y, rows, n, elem_bytes(out_dtype)), {x, rows, k, x_stride, 1}, {w, n, k, w_stride, 1},
                     dense(x_scale, rows, 1, 4), dense(w_scale, n, 1, 4)};
    if (!mats_ok(m, 1)) return GEMM_RELU_EINVAL;
    const RowsPlan r = plan_rows(Linear{rows, n, k, x_stride, w_stride, true, 1});
    if (k > kMaxK8 || r.p.grid() > kMaxGrid) return GEMM_RELU_EUNSUPPORTED;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    auto go = [&](const LinearPlan& p, const Linear& l, int64_t first) {
        KernelArgs a = linear_args(p, l, static_cast<const char*>(x) + first * x_stride, w,
                                   static_cast<char*>(y) + first * n * elem_bytes(out_dtype));
        a.scale_a = x_scale + first;
        a.scale_b = w_scale;
        return launcher_i8(out_dtype, p.cfg)(a, int(p.grid()), st);
    };
    hipError_t e = go(r.p, r.top, 0);
    if (e == hipSuccess && r.rest.M > 0) e = go(r.q, r.rest, r.top.M);
    return finish(e, st);
}

extern "C" const char* gemm_relu_i8_plan(int64_t rows, int64_t n, int64_t k, int out_dtype)
{
    if (!size_ok(rows) || !size_ok(n) || !size_ok(k) || !is_float(out_dtype)) return nullptr;
    if (rows == 0 || n == 0) return "none";
    if (k > kMaxK8) return "unsupported";
    return rows_plan_name(plan_rows(Linear{rows, n, k, k, k, true, 1}));
}
