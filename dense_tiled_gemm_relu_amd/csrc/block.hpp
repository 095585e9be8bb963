// Launch interface of the kernels around the half layer, between the C-ABI unit
// (block_api.hip) and the kernel units.
#pragma once

#include "ffn.hpp"

namespace gemm_relu_hip {

// ---- column sums over strips of rows: out[s][j] = sum over strips of partial[strip][s cols + j]
constexpr int kMaxSums = 4;
struct JoinArgs {
    const float* partial;       // strips x sums x cols
    void* out[kMaxSums];        // null: not wanted
    int sums, cols, strips;
};
hipError_t launch_join(const JoinArgs& a, int out_dt, hipStream_t stream);

// ---- gradient of act(z) (block_rows.hip)
constexpr int kActGradThreads = 512;       // of a workgroup, which takes a 64 x 64 tile
struct ActGradArgs {
    const float* z;             // (rows, n)
    const void* dy;
    void* dz;                   // (rows, n), rows ld apart; null: not wanted
    void* dz_t;                 // (n, rows), rows ld_t apart
    float* sums;                // of dz over each 64 rows (64-row tiles x n); null: not wanted
    int64_t dy_stride;
    int ld, ld_t;
    int rows, n, act;
    float scale;                // of what dz and dz_t hold
    unsigned* flags;            // `nflags` arrival counters to clear for a K split that follows
    int nflags;
};
hipError_t launch_act_grad(const ActGradArgs& a, int dt, hipStream_t stream);

// ---- residual sum and norms (block_rows.hip)
struct AddNormArgs {
    const void* x;
    const void* r;
    const void* gate;           // null: 1
    const void* pw;             // null: x is not normed
    const void* w;              // null: no y
    const void* b;
    void* s;
    void* y;
    float* stats;               // 4 a row: mean and 1 / deviation of x, and of s
    const void* dy;             // backward
    const void* ds;
    void* dx;
    void* dr;
    void* dgate;                // of a gate matrix; the sums over rows go to `partial`
    float* partial;             // strips x 4 x cols: dweight, dbias, dgate, dpost_weight
    float* row_sums;            // 2 a row: the means that dresidual takes (rows of any length)
    int64_t x_stride, r_stride, gate_stride, dy_stride, ds_stride;    // gate_stride 0: one row
    int rows, cols;
    int layer;                  // layer norm, else root mean square
    float scale, eps;
};
hipError_t launch_add_norm(const AddNormArgs& a, int dt, int wdt, hipStream_t stream);
// strips of rows the backward pass sums on their own before launch_join
int add_norm_strips(int64_t rows, int64_t cols, int bytes);
hipError_t launch_add_norm_backward(const AddNormArgs& a, int dt, int wdt, hipStream_t stream);

}  // namespace gemm_relu_hip
