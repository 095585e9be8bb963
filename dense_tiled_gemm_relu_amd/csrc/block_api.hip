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
    const RowsPlan p = plan_rows(Linear{rows, n, k, x_stride, weight_stride, true}, true);
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
    return rows_plan_name(plan_rows(Linear{rows, n, k, k, k, true}, true));
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
    if (p.x.grid() + p.w.grid() + ceil_div(n, 64) > kMaxGrid || ceil_div(n, 64) * ceil_div(rows, 64) * kActGradThreads >= (int64_t(1) << 32))
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
    // dbias in the same launch, behind the products
    const LinearSums sums{reinterpret_cast<const float*>(ws + p.more), dbias, int(n), int(ceil_div(rows, 64)), bias_dtype};
    const int ns = dbias ? int(ceil_div(n, 64)) : 0;
    if (e == hipSuccess && nx + nw + ns > 0) {
        // the product whose tiles take longest first
        const bool x_first = p.lx.K * p.w.splits >= p.lw.K * p.x.splits;
        const LinearPair pair = x_first ? LinearPair{gx, gw, nx} : LinearPair{gw, gx, nw};
        e = launcher_cast_pair_sums(dtype, p.x.cfg)(LinearPairSums{pair, nx + nw, sums}, nx + nw + ns, st);
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

// ------------------------------------------------- residual sum and norms
static bool add_norm_ok(int64_t rows, int64_t cols, int64_t gate_stride, const void* gate, int dtype, int wdtype, int norm,
                        float scale)
{
    return size_ok(rows) && size_ok(cols) && is_float(dtype) && (wdtype == dtype || wdtype == GEMM_RELU_F32) &&
           (norm == GEMM_RELU_NORM_RMS || norm == GEMM_RELU_NORM_LAYER) && scale - scale == 0.0f &&
           (!gate || gate_stride >= 0);
}
// a gate of one row, or a matrix
static Mat gate_matrix(const void* gate, int64_t stride, int64_t rows, int64_t cols, int e, int we)
{
    if (!gate) return dense(nullptr, 0, 0, 1);
    return stride ? Mat{gate, rows, cols, stride, e} : dense(gate, 1, cols, we);
}

extern "C" int gemm_relu_add_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                  const void* gate, int64_t gate_stride, const void* post_weight, const void* weight,
                                  const void* bias, void* s, void* y, float* stats, int64_t rows, int64_t cols, int dtype,
                                  int wdtype, int norm, float scale, float eps, void* stream)
{
    if (!add_norm_ok(rows, cols, gate_stride, gate, dtype, wdtype, norm, scale) || !(eps >= 0.0f) || (rows > 0 && cols < 1) ||
        (!weight && bias))
        return GEMM_RELU_EINVAL;
    if (rows == 0) return GEMM_RELU_OK;
    const int e = elem_bytes(dtype), we = elem_bytes(wdtype);
    const Mat m[] = {dense(s, rows, cols, e), dense(y, weight ? rows : 0, cols, e), dense(stats, stats ? rows : 0, 4, 4),
                     {x, rows, cols, x_stride, e}, {residual, rows, cols, residual_stride, e},
                     gate_matrix(gate, gate_stride, rows, cols, e, we), dense(post_weight, post_weight ? 1 : 0, cols, we),
                     dense(weight, weight ? 1 : 0, cols, we), dense(bias, bias ? 1 : 0, cols, we)};
    if (!mats_ok(m, 3)) return GEMM_RELU_EINVAL;
    if (const int dev = check_device()) return dev;
    AddNormArgs a{};
    a.x = x;
    a.r = residual;
    a.gate = gate;
    a.pw = post_weight;
    a.w = weight;
    a.b = bias;
    a.s = s;
    a.y = y;
    a.stats = stats;
    a.x_stride = x_stride;
    a.r_stride = residual_stride;
    a.gate_stride = gate ? gate_stride : 0;
    a.rows = int(rows);
    a.cols = int(cols);
    a.layer = norm == GEMM_RELU_NORM_LAYER;
    a.scale = scale;
    a.eps = eps;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return finish(launch_add_norm(a, dtype, wdtype, st), st);
}

// the strips' sums, then two sums a row
static uint64_t add_norm_sums(int64_t rows, int64_t cols)
{
    return uint64_t(round_up(int64_t(add_norm_strips(rows)) * kNormSums * cols * 4, 256));
}
extern "C" int64_t gemm_relu_add_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (!size_ok(rows) || !size_ok(cols)) return GEMM_RELU_EINVAL;
    return int64_t(add_norm_sums(rows, cols)) + rows * 2 * 4;
}

extern "C" int gemm_relu_add_norm_backward(const void* dy, int64_t dy_stride, const void* ds, int64_t ds_stride, const void* x,
                                           int64_t x_stride, const void* residual, int64_t residual_stride, const void* gate,
                                           int64_t gate_stride, const void* post_weight, const void* weight,
                                           const float* stats, void* dx, void* dresidual, void* dgate, void* dpost_weight,
                                           void* dweight, void* dbias, int64_t rows, int64_t cols, int dtype, int wdtype,
                                           int norm, float scale, void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (!add_norm_ok(rows, cols, gate_stride, gate, dtype, wdtype, norm, scale) || (rows > 0 && cols < 1) ||
        (!weight && (dweight || dbias)) || (!gate && dgate) || (!post_weight && dpost_weight))
        return GEMM_RELU_EINVAL;
    if (cols == 0) return GEMM_RELU_OK;
    const int e = elem_bytes(dtype), we = elem_bytes(wdtype);
    const uint64_t need = uint64_t(gemm_relu_add_norm_backward_workspace(rows, cols));
    auto vector = [&](const void* p) { return dense(p, p ? 1 : 0, cols, we); };
    auto output = [&](const void* p) { return dense(p, p ? rows : 0, cols, e); };
    const Mat m[] = {output(dx), output(dresidual), gate && gate_stride ? output(dgate) : vector(dgate), vector(dpost_weight),
                     vector(dweight), vector(dbias), bytes_of(workspace, need),
                     weight ? Mat{dy, rows, cols, dy_stride, e} : dense(nullptr, 0, 0, e),
                     ds ? Mat{ds, rows, cols, ds_stride, e} : dense(nullptr, 0, 0, e), {x, rows, cols, x_stride, e},
                     {residual, rows, cols, residual_stride, e}, gate_matrix(gate, gate_stride, rows, cols, e, we),
                     vector(post_weight), vector(weight), dense(stats, rows, 4, 4)};
    if (!mats_ok(m, 7) || !workspace_ok(workspace, workspace_bytes, need)) return GEMM_RELU_EINVAL;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    AddNormArgs a{};
    a.x = x;
    a.r = residual;
    a.gate = gate;
    a.pw = post_weight;
    a.w = weight;
    a.stats = const_cast<float*>(stats);
    a.dy = dy;
    a.ds = ds;
    a.dx = dx;
    a.dr = dresidual;
    a.dgate = dgate;
    a.db = dbias;
    a.partial = static_cast<float*>(workspace);
    a.row_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + add_norm_sums(rows, cols));
    a.x_stride = x_stride;
    a.r_stride = residual_stride;
    a.gate_stride = gate ? gate_stride : 0;
    a.dy_stride = dy_stride;
    a.ds_stride = ds_stride;
    a.rows = int(rows);
    a.cols = int(cols);
    a.layer = norm == GEMM_RELU_NORM_LAYER;
    a.scale = scale;
    hipError_t err = launch_add_norm_backward(a, dtype, wdtype, st);
    void* const row_gate = gate && !gate_stride ? dgate : nullptr;
    if (err == hipSuccess && (dweight || dbias || row_gate || dpost_weight)) {
        JoinArgs j{};
        j.partial = a.partial;
        j.result[0] = {dweight, 0, nullptr, 1.0f};
        j.result[1] = {dbias, 1, nullptr, 1.0f};
        // the third sum is of dresidual norm(x), with a matrix for a gate times it
        j.result[2] = {row_gate, 2, post_weight, scale};
        j.result[3] = {dpost_weight, 2, gate && !gate_stride ? gate : nullptr, scale};
        j.results = kMaxResults;
        j.sums = kNormSums;
        j.cols = int(cols);
        j.strips = add_norm_strips(rows);
        err = launch_join(j, wdtype, st);
    }
    return finish(err, st);
}

// --------------------------------------------------------- orthogonalisation
namespace {

// (the tiles' copies reach rows of 2^22 elements; a launch's work-items stay below 2^32)
constexpr int64_t kOrthoShort = int64_t(1) << 16, kOrthoLong = int64_t(1) << 22, kOrthoSize = int64_t(1) << 34, kOrthoBatch = 65535;
constexpr int64_t kOrthoBatchStride = int64_t(1) << 40;      // more than any memory; what lies behind could wrap
constexpr int kOrthoSteps = int(sizeof(OrthoSteps::v) / (3 * sizeof(float)));

// A symmetric product's configuration, and that of its diagonal tiles where they take a launch
// of their own in smaller tiles (-1: they do not): half of such a tile is wasted, and their few
// can cost a whole round (8192 x 8192, 528 tiles of 256 x 256 on 256 CUs: 560 us; 496 and the
// diagonal 422 + 53).
struct Symmetric {
    int cfg, diagonal;
};
struct OrthoPlan {
    int64_t p, q, P, Q;
    Symmetric gram, poly;                       // configurations of the products
    int step;
    int64_t parts = 1, split_steps = 0;         // of A's K, with LIN_64: steps each
    uint64_t squares, x[2], a, b, diag_a, diag_b, flags, sums, bytes;
};
int64_t triangle(int64_t side) { return side * (side + 1) / 2; }
int64_t side_of(int cfg, const Linear& l) { return ceil_div(l.M, linear_info(cfg).bm); }
// the configurations of least estimated time for `batch` products
int ortho_config(const Linear& l, int64_t batch)
{
    const auto time = [&](int cfg) { return tiles_time(cfg, l, batch * tiles_of(cfg, l)); };
    int best = LIN_64;
    for (int cfg : {LIN_128, LIN_128X2, LIN_256})
        if (usable(cfg, l) && time(cfg) < time(best)) best = cfg;
    return best;
}
int64_t diagonal_tiles(const Symmetric& s, const Linear& l)
{
    return side_of(s.cfg, l) * triangle(linear_info(s.cfg).bm / linear_info(s.diagonal).bm);
}
double symmetric_time(const Symmetric& s, const Linear& l, int64_t batch)
{
    const int64_t side = side_of(s.cfg, l);
    if (s.diagonal < 0) return tiles_time(s.cfg, l, batch * triangle(side));
    return tiles_time(s.cfg, l, batch * triangle(side - 1)) + tiles_time(s.diagonal, l, batch * diagonal_tiles(s, l)) +
           3000.0;                                                                    // a second launch
}
Symmetric symmetric_config(const Linear& l, int64_t batch)
{
    Symmetric best{LIN_64, -1};
    const auto consider = [&](Symmetric s) {
        if (usable(s.cfg, l) && symmetric_time(s, l, batch) < symmetric_time(best, l, batch)) best = s;
    };
    for (int cfg : {LIN_128, LIN_128X2, LIN_256}) {
        consider({cfg, -1});
        if (side_of(cfg, l) > 1)
            for (int diagonal : {LIN_64, LIN_128})
                if (linear_info(diagonal).bm < linear_info(cfg).bm) consider({cfg, diagonal});
    }
    return best;
}
// A = X X^T has the longest K and, of a short X, few tiles: its K is cut into parts where
// the estimate says so (3001 x 1000, 136 tiles of 47 steps: 16 us in one part, 14 in three).  Two
// workgroups that share a CU slow each other down from 0.55 of their time together.
constexpr int kGramParts = 8;
void split_gram(OrthoPlan& o, const Linear& l, int64_t batch)
{
    const int64_t steps = ceil_div(l.K, kSplitStep), tiles = triangle(side_of(LIN_64, l)) * batch;
    const TileTime t = tile_time(LIN_64);
    double best = symmetric_time(o.gram, l, batch);
    for (int64_t parts = 2; parts <= kGramParts; ++parts) {
        if (tiles > kNumCUs || tiles * parts > 2 * kNumCUs || steps < 4 * parts) break;
        const double share = t.alone + (1.0 - t.alone) * double(std::max<int64_t>(0, tiles * parts - kNumCUs)) / kNumCUs;
        const double time = share * (t.per_byte * double(l.K) * l.bytes / double(parts) + t.fixed) + 3000.0;
        if (time >= best) continue;
        best = time;
        o.gram = Symmetric{LIN_64, -1};
        o.split_steps = ceil_div(steps, parts);
        o.parts = ceil_div(steps, o.split_steps);
    }
}
OrthoPlan plan_ortho(int64_t batch, int64_t rows, int64_t cols)
{
    OrthoPlan o{};
    o.p = std::min(rows, cols);
    o.q = std::max(rows, cols);
    o.P = round_up(o.p, 64);
    o.Q = round_up(o.q, 64);
    if (ortho_is_small(o.p, o.q)) return o;
    if (ortho_is_long(batch, o.p, o.q)) {
        const uint64_t parts = uint64_t(ortho_parts(o.q)) * uint64_t(batch), P = uint64_t(o.P);
        o.x[0] = uint64_t(batch) * kOrthoParts * 8;                     // X of the parts' lanes
        o.a = o.x[0] + parts * P * kOrthoPart * 4;                      // two steps' sums
        o.bytes = o.a + 2 * parts * P * P * 4;
        return o;
    }
    o.gram = symmetric_config(Linear{o.P, o.P, o.Q, o.Q, o.Q, true}, batch);
    o.poly = symmetric_config(Linear{o.P, o.P, o.P, o.P, o.P, true}, batch);
    o.step = ortho_config(Linear{o.P, o.Q, 2 * o.P, 2 * o.P, o.Q, false}, batch);
    split_gram(o, Linear{o.P, o.P, o.Q, o.Q, o.Q, true}, batch);
    uint64_t at = 0;
    const auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) & ~uint64_t(255);
        return here;
    };
    const uint64_t PQ = uint64_t(o.P) * uint64_t(o.Q) * uint64_t(batch), PP = uint64_t(o.P) * uint64_t(o.P) * uint64_t(batch);
    o.squares = take(uint64_t(batch) * kOrthoParts * 8);
    o.x[0] = take(PQ * 4);                      // [xl; xh], before a step and after
    o.x[1] = take(PQ * 4);
    o.a = take(PP * 2);
    o.b = take(PP * 4);                         // [B / kLowScale, B]
    o.diag_a = take(uint64_t(o.P) * uint64_t(batch) * 4);
    o.diag_b = take(uint64_t(o.P) * uint64_t(batch) * 4);
    const uint64_t tiles = o.parts > 1 ? uint64_t(triangle(o.P / 64)) * uint64_t(batch) : 0;
    o.flags = take(tiles * 4);
    o.sums = take(tiles * uint64_t(o.parts) * 64 * 64 * 4);
    o.bytes = at;
    return o;
}
bool ortho_sizes_ok(int64_t batch, int64_t rows, int64_t cols) { return size_ok(batch) && size_ok(rows) && size_ok(cols); }
bool ortho_supported(int64_t batch, int64_t rows, int64_t cols)
{
    return batch <= kOrthoBatch && std::min(rows, cols) <= kOrthoShort && std::max(rows, cols) <= kOrthoLong &&
           rows * cols <= kOrthoSize;
}

}  // namespace

extern "C" int64_t gemm_relu_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols)
{
    if (!ortho_sizes_ok(batch, rows, cols)) return GEMM_RELU_EINVAL;
    if (batch == 0 || rows == 0 || cols == 0) return 0;
    if (!ortho_supported(batch, rows, cols)) return GEMM_RELU_EUNSUPPORTED;
    return int64_t(plan_ortho(batch, rows, cols).bytes);
}

extern "C" const char* gemm_relu_orthogonalize_plan(int64_t batch, int64_t rows, int64_t cols)
{
    if (!ortho_sizes_ok(batch, rows, cols)) return nullptr;
    if (batch == 0 || rows == 0 || cols == 0) return "none";
    if (!ortho_supported(batch, rows, cols)) return "unsupported";
    if (ortho_is_small(std::min(rows, cols), std::max(rows, cols))) return "small";
    if (ortho_is_long(batch, std::min(rows, cols), std::max(rows, cols))) return "long";
    // every plan's name, kept for good: three products, of which two may name the tiles on
    // their diagonal, and the first the parts of its K instead (2 to kGramParts)
    constexpr int CFGS = LIN_64 + 1, DIAGONALS = 3, PLAIN = CFGS * DIAGONALS;
    struct Names {
        char text[PLAIN + kGramParts - 1][PLAIN][CFGS][160];
        static int put(char* to, size_t room, int k)
        {
            if (k >= PLAIN) return std::snprintf(to, room, "%s*%d,", linear_info(LIN_64).name, k - PLAIN + 2);
            static constexpr int diagonals[DIAGONALS] = {-1, LIN_128, LIN_64};
            const int d = diagonals[k % DIAGONALS];
            return std::snprintf(to, room, d < 0 ? "%s," : "%s/%s,", linear_info(k / DIAGONALS).name, d < 0 ? "" : linear_info(d).name);
        }
        Names()
        {
            for (int a = 0; a < PLAIN + kGramParts - 1; ++a)
                for (int b = 0; b < PLAIN; ++b)
                    for (int c = 0; c < CFGS; ++c) {
                        char* to = text[a][b][c];
                        size_t at = size_t(put(to, sizeof text[a][b][c], a));
                        at += size_t(put(to + at, sizeof text[a][b][c] - at, b));
                        std::snprintf(to + at, sizeof text[a][b][c] - at, "%s", linear_info(c).name);
                    }
        }
    };
    static const Names names;
    const OrthoPlan o = plan_ortho(batch, rows, cols);
    const auto index = [](const Symmetric& s) { return s.cfg * DIAGONALS + (s.diagonal < 0 ? 0 : s.diagonal == LIN_128 ? 1 : 2); };
    return names.text[o.parts > 1 ? PLAIN + int(o.parts) - 2 : index(o.gram)][index(o.poly)][o.step];
}

extern "C" int gemm_relu_orthogonalize(const void* g, int64_t g_stride, int64_t g_batch_stride, void* out, int64_t batch,
                                       int64_t rows, int64_t cols, int dtype, const float* coefficients, int steps, float eps,
                                       void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (!ortho_sizes_ok(batch, rows, cols) || !is_float(dtype) || steps < 0 || steps > kOrthoSteps || (steps > 0 && !coefficients) ||
        !(eps >= 0.0f) || g_batch_stride < 0 || g_batch_stride > kOrthoBatchStride)
        return GEMM_RELU_EINVAL;
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_RELU_OK;
    if (!ortho_supported(batch, rows, cols)) return GEMM_RELU_EUNSUPPORTED;
    const OrthoPlan o = plan_ortho(batch, rows, cols);
    const int e = elem_bytes(dtype);
    // the batch's matrices may lie in any order and overlap; the last one ends the furthest
    Mat in{g, rows, cols, g_stride, e};
    if (!in.ok()) return GEMM_RELU_EINVAL;
    const uint64_t span = uint64_t(batch - 1) * uint64_t(g_batch_stride) * uint64_t(e) + in.span();
    const uint64_t out_bytes = uint64_t(batch) * uint64_t(rows) * uint64_t(cols) * 2;
    const uintptr_t at = reinterpret_cast<uintptr_t>(out), ws_at = reinterpret_cast<uintptr_t>(workspace);
    if (!out || (at & 1) || overlaps(at, out_bytes, in.at(), span) || overlaps(at, out_bytes, ws_at, o.bytes) ||
        overlaps(ws_at, o.bytes, in.at(), span) || !workspace_ok(workspace, workspace_bytes, o.bytes))
        return GEMM_RELU_EINVAL;
    for (int k = 0; k < 3 * steps; ++k)
        if (!(coefficients[k] - coefficients[k] == 0.0f)) return GEMM_RELU_EINVAL;
    if (const int dev = check_device()) return dev;
    hipStream_t st = static_cast<hipStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    OrthoArgs a{};
    a.g = g;
    a.g_stride = g_stride;
    a.g_batch = g_batch_stride;
    a.out = out;
    a.rows = int(rows);
    a.cols = int(cols);
    a.batch = int(batch);
    a.p = int(o.p);
    a.q = int(o.q);
    a.P = int(o.P);
    a.Q = int(o.Q);
    a.eps = eps;
    a.squares = reinterpret_cast<double*>(ws + o.squares);
    a.parts = ortho_square_parts(rows, cols, dtype);
    const uint64_t PQ = uint64_t(o.P) * uint64_t(o.Q), PP = uint64_t(o.P) * uint64_t(o.P);
    a.xl = ws + o.x[0];
    a.xh = ws + o.x[0] + PQ * 2;
    const int64_t gram_tiles = triangle(o.P / 64);             // of a cut product
    a.flags = reinterpret_cast<unsigned*>(ws + o.flags);
    a.nflags = o.parts > 1 ? int(gram_tiles) : 0;
    const bool small = ortho_is_small(o.p, o.q);
    if (small || ortho_is_long(batch, o.p, o.q)) {
        OrthoSteps c{};
        c.steps = steps;
        std::copy_n(coefficients, 3 * steps, c.v);
        float *const x = reinterpret_cast<float*>(ws + o.x[0]), *const sums = reinterpret_cast<float*>(ws + o.a);
        return finish(small ? launch_ortho_small(a, c, dtype, st) : launch_ortho_long(a, c, x, sums, dtype, st), st);
    }
    hipError_t err = launch_ortho_start(a, dtype, st);
    const Linear gram{o.P, o.P, o.Q, o.Q, o.Q, true}, poly{o.P, o.P, o.P, o.P, o.P, true}, next{o.P, o.Q, 2 * o.P, 2 * o.P, o.Q, false};
    const auto product = [&](int cfg, const Linear& l, const void* A, const void* B, void* C) {
        OrthoProduct k{};
        k.k = linear_args(plan_as(cfg, l), l, A, B, C);
        k.k.split_steps = int(ceil_div(l.K, kSplitStep));      // one part, where the configuration can cut K
        k.diag = uint64_t(o.P);
        return k;
    };
    // a symmetric product in one launch, or its tiles below the diagonal and then those on it
    const auto symmetric = [&](int epi, const Symmetric& c, const Linear& l, OrthoProduct k) {
        const int64_t side = side_of(c.cfg, l);
        if (c.diagonal < 0) return launcher_ortho(epi, c.cfg)(k, int(triangle(side)) * k.k.splits, int(batch), st);
        k.k.triangle = 1;
        const hipError_t e = launcher_ortho(epi, c.cfg)(k, int(triangle(side - 1)), int(batch), st);
        if (e != hipSuccess) return e;
        k.k.triangle = 2;
        k.k.sub = linear_info(c.cfg).bm / linear_info(c.diagonal).bm;
        k.k.tiles_m = k.k.tiles_n = int(side_of(c.diagonal, l));
        return launcher_ortho(epi, c.diagonal)(k, int(diagonal_tiles(c, l)), int(batch), st);
    };
    for (int s = 0; s < steps && err == hipSuccess; ++s) {
        const unsigned char *const xl = ws + o.x[s % 2], *const xh = xl + PQ * 2;
        unsigned char* const to = ws + o.x[(s + 1) % 2];
        const bool last = s == steps - 1;
        OrthoProduct k = product(o.gram.cfg, gram, xh, xh, ws + o.a);
        k.k.alpha = kOrthoA / (kOrthoX * kOrthoX);
        k.k.beta = 1.0f / (kOrthoX * kOrthoX);
        k.k.diag = reinterpret_cast<float*>(ws + o.diag_a);
        k.a = k.b = PQ * 4;
        k.c = PP * 2;
        if (o.parts > 1) {
            k.k.splits = int(o.parts);
            k.k.split_steps = int(o.split_steps);
            k.k.ws = reinterpret_cast<float*>(ws + o.sums);
            k.k.flags = a.flags;
            k.ws = uint64_t(gram_tiles) * uint64_t(o.parts) * 64 * 64;
            k.flags = uint64_t(gram_tiles);
        }
        err = symmetric(EPI_GRAM, o.gram, gram, k);
        if (err != hipSuccess) break;
        k = product(o.poly.cfg, poly, ws + o.a, ws + o.a, ws + o.b);
        k.k.alpha = kOrthoB;
        k.k.beta = 1.0f / (kOrthoA * kOrthoA);
        k.k.scale_o = 1.0f / kOrthoA;
        k.k.pb = coefficients[3 * s + 1];
        k.k.pc = coefficients[3 * s + 2];
        k.k.diag = reinterpret_cast<float*>(ws + o.diag_a);
        k.k.diag_out = reinterpret_cast<float*>(ws + o.diag_b);
        k.k.R = ws + o.a;
        k.k.ldr = int(o.P);
        k.a = k.b = k.r = PP * 2;
        k.c = PP * 4;
        err = symmetric(EPI_POLY, o.poly, poly, k);
        if (err != hipSuccess) break;
        // [B / kLowScale, B] [xl; xh]
        k = product(o.step, next, ws + o.b, xl, last ? out : to + PQ * 2);
        k.k.alpha = 1.0f / kOrthoX;             // of the last step's result
        k.k.beta = 1.0f / kOrthoB;
        k.k.pa = coefficients[3 * s];
        k.k.diag = reinterpret_cast<float*>(ws + o.diag_b);
        k.k.R = xh;
        k.k.L = xl;
        k.k.low = to;
        k.k.ldr = int(o.Q);
        k.k.out_m = int(o.p);
        k.k.out_n = int(o.q);
        k.k.transposed = rows > cols;
        k.a = PP * 4;
        k.b = k.r = k.low = PQ * 4;
        k.c = last ? uint64_t(rows) * uint64_t(cols) * 2 : PQ * 4;
        err = launcher_ortho(last ? EPI_LAST : EPI_STEP, o.step)(k, int(tiles_of(o.step, next)), int(batch), st);
    }
    if (err == hipSuccess && steps == 0) err = launch_ortho_copy(a, st);
    return finish(err, st);
}
