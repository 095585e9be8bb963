// Launch interface of the kernels around the half layer, between the C-ABI unit
// (block_api.hip) and the kernel units.
#pragma once

#include "ffn.hpp"

namespace gemm_relu_hip {

// ---- column sums over strips of rows: out[s][j] = sum over strips of partial[strip][s cols + j]
constexpr int kMaxSums = 5;
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

}  // namespace gemm_relu_hip
