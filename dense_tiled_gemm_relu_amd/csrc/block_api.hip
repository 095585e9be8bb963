// C-ABI of the operators around the half layer (include/gemm_relu_block.h): argument
// checks, configuration choice, launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_common.hpp"
#include "block.hpp"
#include "gemm_relu_block.h"
#include "linear_plan.hpp"

using namespace gemm_relu_hip;

// ------------------------------------- product with bias, activation, residual
static bool act_sizes_ok(int64_t rows, int64_t n, int64_t k, int dtype)
{
    return size_ok(rows) && size_ok(n) && size_ok(k) && is_16bit(dtype);
}
static bool act_codes_ok(int dtype, int bias_dtype, int act)
{
    return (bias_dtype == dtype || bias_dtype == GEMM_RELU_F32) && act >= GEMM_RELU_ACT_SILU && act <= GEMM_RELU_ACT_NONE;
}

extern "C" int gemm_relu_act(const void* x, int64_t x_stride, const void* weight, int64_t weight_stride,
                             const void* bias, const void* residual, int64_t residual_stride, void* y, float* z,
                             int64_t rows, int64_t n, int64_t k, int dtype, int bias_dtype, int act, void* stream)
{
    if (!act_sizes_ok(rows, n, k, dtype) || !act_codes_ok(dtype, bias_dtype, act)) return GEMM_RELU_EINVAL;
    if (rows == 0 || n == 0) return GEMM_RELU_OK;
    const Mat r = residual ? Mat{residual, rows, n, residual_stride, 2} : dense(nullptr, 0, 0, 2);
    const Mat m[] = {dense(y, rows, n, 2), dense(z, z ? rows : 0, n, 4), {x, rows, k, x_stride, 2},
                     {weight, n, k, weight_stride, 2}, dense(bias, bias ? 1 : 0, n, elem_bytes(bias_dtype)), r};
    if (!mats_ok(m, 2)) return GEMM_RELU_EINVAL;
    const RowsPlan p = plan_rows(Linear{rows, n, k, x_stride, weight_stride, true});
    if (k > kMaxK || p.p.grid() > kMaxGrid) return GEMM_RELU_EUNSUPPORTED;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    auto go = [&](const LinearPlan& q, const Linear& l, int64_t first) {
        KernelArgs a = linear_args(q, l, static_cast<const char*>(x) + 2 * first * x_stride, weight,
                                   static_cast<char*>(y) + 2 * first * n);
        a.act = act;
        a.GU = z ? z + first * n : nullptr;
        a.bias = bias;
        a.bias_f32 = bias_dtype == GEMM_RELU_F32;
        a.ldr = int(r.stride);
        a.R = residual ? static_cast<const unsigned char*>(residual) + 2 * first * residual_stride : nullptr;
        return launcher_act(dtype, q.cfg)(a, int(q.grid()), st);
    };
    hipError_t e = go(p.p, p.top, 0);
    if (e == hipSuccess && p.rest.M > 0) e = go(p.q, p.rest, p.top.M);
    return finish(e, st);
}

extern "C" const char* gemm_relu_act_plan(int64_t rows, int64_t n, int64_t k, int dtype)
{
    if (!act_sizes_ok(rows, n, k, dtype)) return nullptr;
    if (rows == 0 || n == 0) return "none";
    if (k > kMaxK) return "unsupported";
    return rows_plan_name(plan_rows(Linear{rows, n, k, k, k, true}));
}

// the products' plan, behind whose workspace the sums of dz over each 64 rows lie
static GradPlan plan_act_grad(int64_t rows, int64_t n, int64_t k, int64_t x_stride, int64_t weight_stride)
{
    return plan_grad(rows, n, k, x_stride, weight_stride, uint64_t(ceil_div(rows, 64)) * uint64_t(n) * 4);
}

extern "C" int64_t gemm_relu_act_backward_workspace(int64_t rows, int64_t n, int64_t k)
{
    if (!act_sizes_ok(rows, n, k, GEMM_RELU_F16)) return GEMM_RELU_EINVAL;
    if (rows > kMaxGradRows || n > kMaxGradRows) return GEMM_RELU_EUNSUPPORTED;
    return int64_t(plan_act_grad(rows, n, k, k, k).bytes);
}

extern "C" int gemm_relu_act_backward(const void* dy, int64_t dy_stride, const float* z, const void* x, int64_t x_stride,
                                      const void* weight, int64_t weight_stride, void* dx, void* dweight, void* dbias,
                                      int64_t rows, int64_t n, int64_t k, int dtype, int bias_dtype, int act,
                                      void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (!act_sizes_ok(rows, n, k, dtype) || !act_codes_ok(dtype, bias_dtype, act)) return GEMM_RELU_EINVAL;
    if (n == 0 && (rows == 0 || k == 0)) return GEMM_RELU_OK;
    if (k == 0 && !dbias) return GEMM_RELU_OK;
    if (rows > kMaxGradRows || n > kMaxGradRows) return GEMM_RELU_EUNSUPPORTED;
    const GradPlan p = plan_act_grad(rows, n, k, x_stride, weight_stride);
    const bool slopes = act != GEMM_RELU_ACT_NONE;
    const Mat m[] = {dense(dx, rows, k, 2), dense(dweight, n, k, 2), dense(dbias, dbias ? 1 : 0, n, elem_bytes(bias_dtype)),
                     bytes_of(workspace, p.bytes), {dy, rows, n, dy_stride, 2}, dense(z, slopes ? rows : 0, n, 4),
                     {x, rows, k, x_stride, 2}, {weight, n, k, weight_stride, 2}};
    if (!mats_ok(m, 4) || !workspace_ok(workspace, workspace_bytes, p.bytes)) return GEMM_RELU_EINVAL;
    if (p.x.grid() + p.w.grid() > kMaxGrid || ceil_div(n, 64) * ceil_div(rows, 64) * kActGradThreads >= (int64_t(1) << 32))
        return GEMM_RELU_EUNSUPPORTED;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    unsigned* flags = reinterpret_cast<unsigned*>(ws + p.flags);
    // dy itself is dx's operand where there is no activation and no piece of 16 bytes
    // crosses the end of a row (whole K steps, or dense rows of whole pieces)
    Linear lx = p.lx;
    const void* dz = ws;
    const bool direct = !slopes && dy_stride <= (int64_t(1) << 22) && (n % 64 == 0 || (n % 8 == 0 && dy_stride == n));
    if (direct) {
        lx.lda = dy_stride;
        dz = dy;
    }
    // slopes of these activations reach 1.13: half of a float16 dz is within range
    const bool halve = dtype == GEMM_RELU_F16 && slopes && act != GEMM_RELU_ACT_RELU;
    hipError_t e = hipSuccess;
    if (rows > 0 && n > 0) {
        ActGradArgs g{};
        g.z = z;
        g.dy = dy;
        g.dz = direct ? nullptr : ws;
        g.dz_t = ws + p.dz_t;
        g.sums = dbias ? reinterpret_cast<float*>(ws + p.more) : nullptr;
        g.dy_stride = dy_stride;
        g.ld = int(p.lx.lda);
        g.ld_t = int(p.lw.lda);
        g.rows = int(rows);
        g.n = int(n);
        g.act = act;
        g.scale = halve ? 0.5f : 1.0f;
        g.flags = flags;
        g.nflags = p.nflags();
        e = launch_act_grad(g, dtype, st);
    }
    KernelArgs gx = linear_args(p.x, lx, dz, weight, dx), gw = linear_args(p.w, p.lw, ws + p.dz_t, x, dweight);
    gx.alpha = gw.alpha = halve ? 2.0f : 1.0f;
    gx.flags = flags;
    gx.ws = reinterpret_cast<float*>(ws + p.sums_x);
    gw.flags = flags + (p.x.splits > 1 ? p.x.tiles() : 0);
    gw.ws = reinterpret_cast<float*>(ws + p.sums_w);
    const int nx = rows > 0 && k > 0 ? int(p.x.grid()) : 0, nw = n > 0 && k > 0 ? int(p.w.grid()) : 0;
    if (e == hipSuccess && nx + nw > 0) {
        // the product whose tiles take longest first
        const bool x_first = p.lx.K * p.w.splits >= p.lw.K * p.x.splits;
        e = launcher_cast_pair(dtype, p.x.cfg)(x_first ? LinearPair{gx, gw, nx} : LinearPair{gw, gx, nw}, nx + nw, st);
    }
    if (e == hipSuccess && dbias && n > 0) {
        JoinArgs j{};
        j.partial = reinterpret_cast<const float*>(ws + p.more);
        j.out[0] = dbias;
        j.sums = 1;
        j.cols = int(n);
        j.strips = int(ceil_div(rows, 64));
        e = launch_join(j, bias_dtype, st);
    }
    return finish(e, st);
}

extern "C" const char* gemm_relu_act_backward_plan(int64_t rows, int64_t n, int64_t k, int dtype)
{
    if (!act_sizes_ok(rows, n, k, dtype)) return nullptr;
    if (k == 0 || (rows == 0 && n == 0)) return "none";
    if (rows > kMaxGradRows || n > kMaxGradRows) return "unsupported";
    const GradPlan p = plan_act_grad(rows, n, k, k, k);
    static const PairNames names(',');
    return names.text[p.x.cfg][p.w.cfg];
}
