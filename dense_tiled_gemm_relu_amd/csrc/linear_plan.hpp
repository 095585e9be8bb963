// Matrix arguments and the choice of a product's configuration, shared by the C-ABI
// units.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "api_common.hpp"
#include "ffn.hpp"
#include "gemm_relu.h"

namespace gemm_relu_hip {

namespace {

constexpr int64_t kLim = INT32_MAX;

int elem_bytes(int dt) { return dt == GEMM_RELU_F32 ? 4 : dt == DT_I8 ? 1 : 2; }
bool is_16bit(int dt) { return dt == GEMM_RELU_F16 || dt == GEMM_RELU_BF16; }
bool is_float(int dt) { return is_16bit(dt) || dt == GEMM_RELU_F32; }
bool size_ok(int64_t n) { return n >= 0 && n <= kLim; }

// A matrix argument: rows x cols elements of `bytes` bytes, rows `stride` apart.
struct Mat {
    const void* p;
    int64_t rows, cols, stride;
    int bytes;
    uintptr_t at() const { return reinterpret_cast<uintptr_t>(p); }
    uint64_t span() const
    {
        return rows == 0 || cols == 0 ? 0 : (uint64_t(rows - 1) * uint64_t(stride) + uint64_t(cols)) * uint64_t(bytes);
    }
    bool ok() const { return stride >= cols && stride <= kLim && !(span() && !p) && !(at() & uintptr_t(bytes - 1)); }
};
Mat dense(const void* p, int64_t rows, int64_t cols, int bytes) { return Mat{p, rows, cols, cols, bytes}; }

// Whether every matrix is well formed and no output (the first `outs`)
// overlaps another matrix.
template <size_t N> bool mats_ok(const Mat (&m)[N], size_t outs)
{
    for (size_t i = 0; i < N; ++i)
        if (!m[i].ok()) return false;
    for (size_t i = 0; i < outs; ++i)
        for (size_t j = i + 1; j < N; ++j)
            if (m[i].p && m[j].p && overlaps(m[i].at(), m[i].span(), m[j].at(), m[j].span())) return false;
    return true;
}

// A workspace as a matrix of bytes (256-byte alignment is checked apart).
Mat bytes_of(const void* p, uint64_t n) { return Mat{p, int64_t(n), 1, 1, 1}; }
bool workspace_ok(const void* ws, uint64_t have, uint64_t need)
{
    return need == 0 || (ws && have >= need && !(reinterpret_cast<uintptr_t>(ws) & 255));
}

int finish(hipError_t e, hipStream_t st)
{
    if (e != hipSuccess) return GEMM_RELU_EHIP;
    const char* s = std::getenv("GEMM_RELU_SYNC");
    if (s && s[0] == '1') {
        if (hipStreamSynchronize(st) != hipSuccess) return GEMM_RELU_EHIP;
        if (hipGetLastError() != hipSuccess) return GEMM_RELU_EHIP;
    }
    return GEMM_RELU_OK;
}

// ---- matrix products: C (M x N) = A op(B) over K, element rows lda and ldb apart
struct Linear {
    int64_t M, N, K, lda, ldb;
    bool trans;             // B stored (N,K); else (K,N)
    int bytes = 2;          // of an element of A and B
};
struct LinearPlan {
    int cfg = LIN_G64;
    int64_t tiles_m = 0, tiles_n = 0;
    int64_t splits = 1, split_steps = 0;   // LIN_64 with B stored (K,N): parts of K, steps each
    int64_t tiles() const { return tiles_m * tiles_n; }
    int64_t grid() const { return tiles() * splits; }
};

// Estimated times, in ns, from measurements of each configuration between 1 and
// 14 rounds of workgroups, K from 250 to 16384 and 16-bit and 8-bit inputs (the
// bytes of K count: what bounds the small tiles is the rate at which the L2 feeds
// the copies, 11-12 TB/s, and the largest tile's matrix rate scales alike).
struct TileTime {
    double per_byte, fixed;   // of a tile, per byte of K and for its start and end
    int slots;                // tiles in flight on the device
    double alone;             // share of that time where a CU holds one of two possible tiles
};
TileTime tile_time(int cfg)
{
    switch (cfg) {
    case LIN_256: return {12.0, 4000, kNumCUs, 1.0};
    case LIN_128: return {4.6, 2500, kNumCUs, 1.0};
    case LIN_128X2: return {8.5, 3200, 2 * kNumCUs, 0.75};
    case LIN_64: return {5.2, 2000, 2 * kNumCUs, 0.55};
    case LIN_K16: return {1.2, 1000, 2 * kNumCUs, 0.6};
    case LIN_K32: return {1.4, 800, kNumCUs, 1.0};
    case LIN_K32X48:
    case LIN_K48X32: return {1.75, 900, kNumCUs, 1.0};
    case LIN_K64X32: return {2.0, 900, kNumCUs, 1.0};
    default: return {15.0, 4000, 2 * kNumCUs, 0.6};      // LIN_G64
    }
}
int64_t tiles_of(int cfg, const Linear& l)
{
    return ceil_div(l.M, linear_info(cfg).bm) * ceil_div(l.N, linear_info(cfg).bn);
}
double tiles_time(int cfg, const Linear& l, int64_t tiles)
{
    const TileTime t = tile_time(cfg);
    const double one = t.per_byte * double(l.K) * l.bytes + t.fixed;
    const int64_t rest = tiles % t.slots;
    return one * double(tiles / t.slots) + (rest == 0 ? 0.0 : rest <= kNumCUs ? t.alone * one : one);
}

double linear_time(int cfg, const Linear& l) { return tiles_time(cfg, l, tiles_of(cfg, l)); }

// Whether a configuration can take a product: the tiles' copies have 32-bit
// offsets (256 rows of A, or of B stored (N,K), or a K step's rows of B stored
// (K,N), whose last tile column ends at N); the LIN_K* forms have no such limit.
bool usable(int cfg, const Linear& l)
{
    if (cfg == LIN_G64) return true;
    if (cfg >= LIN_K16) return l.trans && l.K * l.bytes >= 16 && l.K * l.bytes <= (int64_t(1) << 30);
    return l.lda <= (int64_t(1) << 22) && l.ldb <= (int64_t(1) << (l.trans ? 22 : 24)) &&
           (l.trans || l.N >= linear_info(cfg).bn);
}

LinearPlan plan_as(int cfg, const Linear& l)
{
    LinearPlan p;
    p.cfg = cfg;
    p.tiles_m = ceil_div(l.M, linear_info(cfg).bm);
    p.tiles_n = ceil_div(l.N, linear_info(cfg).bn);
    return p;
}

// The configuration of least estimated time; equal ones go to the smaller tile.  The
// register-staged tile is never the fastest but where rows are too far apart for the
// other tiles and K is short (1024 x 512 x 32 gated, rows 2^22 + 8 apart, 5.9 us, 9.3 on
// 32 x 32; 1024 x 512 x 512 14.2 and 11.3).
LinearPlan plan_linear(const Linear& l, bool k64x32 = false)
{
    int best = LIN_G64;
    for (int cfg : {LIN_K16, LIN_K32, LIN_K32X48, LIN_K48X32, LIN_K64X32, LIN_64, LIN_128, LIN_128X2, LIN_256})
        if ((cfg != LIN_K64X32 || k64x32) && usable(cfg, l) && linear_time(cfg, l) < linear_time(best, l)) best = cfg;
    return plan_as(best, l);
}

// Workgroups a product's launch may have: a launch's work-items have to stay below
// 2^32, and a workgroup has up to 512.
constexpr int64_t kMaxGrid = int64_t(1) << 22;

// A product with B stored (N,K) whose last tile row holds a few rows only: these
// go to a launch of their own with small tiles where the estimate says so, since
// the row of mostly empty tiles can cost a whole round (gated 1027 x 2003 x 1501:
// 38 us in one launch).
struct RowsPlan {
    Linear top, rest;
    LinearPlan p, q;            // q: of the rest, if it has rows
};
constexpr int64_t kRestRows = 32;
RowsPlan plan_rows(const Linear& l, bool k64x32 = false)
{
    RowsPlan r{l, l, plan_linear(l, k64x32), {}};
    r.rest.M = 0;
    double best = linear_time(r.p.cfg, l);
    for (int cfg : {LIN_128, LIN_128X2, LIN_256}) {
        Linear top = l, rest = l;
        rest.M = l.M % linear_info(cfg).bm;
        top.M = l.M - rest.M;
        if (top.M == 0 || rest.M == 0 || rest.M > kRestRows || !usable(cfg, l)) continue;
        const LinearPlan q = plan_linear(rest, k64x32);
        if (q.grid() > kMaxGrid) continue;
        const double t = linear_time(cfg, top) + linear_time(q.cfg, rest) + 3000.0;    // a second launch
        if (t < best) {
            r = RowsPlan{top, rest, plan_as(cfg, top), q};
            best = t;
        }
    }
    return r;
}
// Names of two configurations with `between` between them, kept for good.
struct PairNames {
    char text[LIN_COUNT][LIN_COUNT][64];
    explicit PairNames(char between)
    {
        for (int a = 0; a < LIN_COUNT; ++a)
            for (int b = 0; b < LIN_COUNT; ++b)
                std::snprintf(text[a][b], sizeof text[a][b], "%s%c%s", linear_info(a).name, between, linear_info(b).name);
    }
};
const char* rows_plan_name(const RowsPlan& r)
{
    static const PairNames names('+');
    return r.rest.M == 0 ? linear_info(r.p.cfg).name : names.text[r.p.cfg][r.q.cfg];
}

KernelArgs linear_args(const LinearPlan& p, const Linear& l, const void* A, const void* B, void* C)
{
    KernelArgs a{};
    a.A = static_cast<const unsigned char*>(A);
    a.B = static_cast<const unsigned char*>(B);
    a.C = static_cast<unsigned char*>(C);
    a.M = int(l.M);
    a.N = int(l.N);
    a.K = int(l.K);
    a.lda = int(l.lda);
    a.ldb = int(l.ldb);
    a.tiles_m = int(p.tiles_m);
    a.tiles_n = int(p.tiles_n);
    a.splits = int(p.splits);
    a.split_steps = int(p.split_steps);
    a.panel = int(std::min<int64_t>(8, p.tiles_m));
    a.nxcd = 8;
    a.alpha = 1.0f;
    return a;
}

int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// The backward pass of projections onto `outs` columns (the gated ones have 2 hidden): the
// gradients of their sums go to the workspace row-major (rows of outs) for dx, and
// transposed (rows of `rows`) for dweight, each row padded to 16 bytes.  Both products
// share one launch, and so one configuration: dx alone seldom fills the device.  Where
// one of them has few tiles and a long K, its K is cut into parts, whose fp32 sums and
// arrival counters follow in the workspace, and last `more` bytes for the element-wise
// pass.
struct GradPlan {
    Linear lx, lw;
    LinearPlan x, w;            // of dx = dz weight and of dweight = dz^T x
    uint64_t dz_t, flags, sums_x, sums_w, more, bytes;
    int nflags() const { return int((x.splits > 1 ? x.tiles() : 0) + (w.splits > 1 ? w.tiles() : 0)); }
};
// of dx and of dweight: a launch of the largest tiles has no room for more (and the
// workspace's size stays below 2^63)
constexpr int64_t kMaxGradRows = kMaxGrid * 256;
constexpr int64_t kSplitStep = 64;         // K elements per step of LIN_64

// p cut into `parts` of whole steps; false where that leaves a part under 4 steps
bool split(LinearPlan& p, const Linear& l, int64_t parts)
{
    const int64_t steps = ceil_div(l.K, kSplitStep);
    if (parts > 1 && (steps < 4 * parts || p.tiles() > kNumCUs)) return false;
    p.split_steps = steps == 0 ? 1 : ceil_div(steps, parts);
    p.splits = steps == 0 ? 1 : ceil_div(steps, p.split_steps);
    return true;
}
double pair_time(const LinearPlan& p, const Linear& a, const LinearPlan& q, const Linear& b)
{
    const TileTime t = tile_time(p.cfg);
    // a part exchanges its sums through memory, about 3 us
    auto one = [&](const LinearPlan& p, const Linear& l) {
        return t.per_byte * double(l.K) * l.bytes / double(p.splits) + t.fixed + (p.splits > 1 ? 3000.0 : 0.0);
    };
    const double one_a = one(p, a), one_b = one(q, b);
    const double alone = p.grid() + q.grid() <= kNumCUs ? t.alone : 1.0;
    return std::max((one_a * double(p.grid()) + one_b * double(q.grid())) / t.slots + 0.5 * std::min(one_a, one_b),
                    alone * std::max(one_a, one_b));
}
GradPlan plan_grad(int64_t rows, int64_t outs, int64_t cols, int64_t x_stride, int64_t weight_stride, uint64_t more)
{
    GradPlan g;
    const int64_t ld = round_up(outs, 8), ld_t = round_up(rows, 8);
    g.lx = Linear{rows, cols, outs, ld, weight_stride, false};
    g.lw = Linear{outs, cols, rows, ld_t, x_stride, false};
    g.x = plan_as(LIN_G64, g.lx);
    g.w = plan_as(LIN_G64, g.lw);
    double best = 0.0;
    auto consider = [&](int cfg, int64_t parts_x, int64_t parts_w) {
        LinearPlan x = plan_as(cfg, g.lx), w = plan_as(cfg, g.lw);
        if (cfg == LIN_64 && !(split(x, g.lx, parts_x) && split(w, g.lw, parts_w))) return;
        const double t = pair_time(x, g.lx, w, g.lw);
        if (g.x.cfg != LIN_G64 && t >= best) return;
        g.x = x;
        g.w = w;
        best = t;
    };
    for (int cfg : {LIN_64, LIN_128, LIN_128X2, LIN_256})
        if (usable(cfg, g.lx) && usable(cfg, g.lw)) consider(cfg, 1, 1);
    if (usable(LIN_64, g.lx) && usable(LIN_64, g.lw) && rows > 0 && outs > 0)
        for (int64_t parts : {2, 4, 8, 16}) {
            consider(LIN_64, parts, 1);
            consider(LIN_64, 1, parts);
        }
    auto sums = [](const LinearPlan& p) { return p.splits > 1 ? uint64_t(p.grid()) * 64 * 64 * 4 : 0; };
    g.dz_t = uint64_t(round_up(2 * rows * ld, 256));
    g.flags = uint64_t(round_up(int64_t(g.dz_t + uint64_t(outs) * uint64_t(ld_t) * 2), 256));
    g.sums_x = g.flags + uint64_t(round_up(4 * int64_t(g.nflags()), 256));
    g.sums_w = g.sums_x + sums(g.x);
    g.more = g.sums_w + sums(g.w);
    g.bytes = g.more + more;
    return g;
}

}  // namespace

}  // namespace gemm_relu_hip
