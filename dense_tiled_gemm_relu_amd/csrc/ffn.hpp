// Launch interface of the feed-forward operators' kernels, between the C-ABI
// unit (ffn_api.hip) and the kernel units.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_relu_kernel.hpp"

namespace gemm_relu_hip {

// 1 KiB, 16 bytes a lane from any address, to LDS bytes lds .. lds + 1023 in lane
// order; no register holds it on the way, so it is waited for with vmcnt.
__device__ __forceinline__ void copy_to_lds(const unsigned char* from, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\t"
                 "s_nop 0\n\t"
                 "global_load_lds_dwordx4 %0, off"
                 :
                 : "v"(from), "s"(lds)
                 : "memory", "m0");
}

// ---- matrix products (inst_ffn.hip)
// The tiles of the GEMM + ReLU, with the epilogues of the feed-forward operators;
// BK in a name counts 16-bit elements, as there.  LIN_128 has four stages and a
// CU to itself, LIN_128X2 two and half a CU, LIN_64 four and half a CU; with B
// stored (K,N), LIN_64 can cut a tile's K into parts.  LIN_K16 and the others of
// ffn_skinny.hip (K cut between a workgroup's waves) serve only products with B
// stored (N,K).
enum LinearConfig : int { LIN_256 = 0, LIN_128, LIN_128X2, LIN_64, LIN_G64, LIN_K16, LIN_K32, LIN_K32X48, LIN_K48X32, LIN_COUNT };

struct LinearInfo {
    const char* name;
    int bm, bn;
};

inline const LinearInfo& linear_info(int cfg)
{
    static const LinearInfo table[LIN_COUNT] = {
        {"d256x256x32_s4_i16w8", 256, 256}, {"d128x128x64_s4_i16w8", 128, 128}, {"d128x128x64_s2w8", 128, 128},
        {"d64x64x64_s4", 64, 64},           {"g64x64x64", 64, 64},              {"k16x16x64_s4", 16, 16},
        {"k32x32x64_s4", 32, 32},           {"k32x48x64_s3", 32, 48},       {"k48x32x64_s3", 48, 32},
    };
    return table[cfg];
}

typedef hipError_t (*LinearLaunchFn)(const KernelArgs& args, int grid, hipStream_t stream);
// two products (either may be empty), B stored (K,N), of one configuration in one launch: `first` workgroups of a, then b's
struct LinearPair {
    KernelArgs a, b;
    int first;
};
typedef hipError_t (*PairLaunchFn)(const LinearPair& pair, int grid, hipStream_t stream);
PairLaunchFn launcher_cast_pair(int dt, int cfg);
LinearLaunchFn launcher_gated(int dt, int cfg);                // B stored (N,K)
LinearLaunchFn launcher_i8(int out_dt, int cfg);               // B stored (N,K)
LinearLaunchFn launcher_skinny_gated(int dt, int cfg);         // the LIN_K* forms of both
LinearLaunchFn launcher_skinny_i8(int out_dt, int cfg);

// ---- rows and element-wise work (ffn_rows.hip)
struct NormArgs {
    const void* x;
    const void* w;
    const void* b;          // null: zero
    void* y;
    float* mean;            // null: not wanted (forward)
    float* rstd;
    const void* dy;         // backward
    void* dx;
    void* dw;
    void* db;               // null: not wanted
    float* partial;         // backward: per strip, cols sums for dw, then cols for db
    int64_t x_stride, dy_stride;
    int rows, cols;
    float eps;
};
hipError_t launch_layer_norm(const NormArgs& a, int dt, int wdt, hipStream_t stream);
// strips of rows the backward pass sums on their own before joining them
// (bytes: of an element of x)
int layer_norm_strips(int64_t rows, int64_t cols, int bytes);
hipError_t launch_layer_norm_backward(const NormArgs& a, int dt, int wdt, hipStream_t stream);

constexpr int kGradThreads = 512;          // of a workgroup, which takes a 64 x 64 tile
// What a tile of dg and du holds past float16's largest value, a bit each: its rows,
// its units of dg and its units of du.
typedef unsigned long long GradMask;
struct GatedGradArgs {
    const float* gu;        // (rows, 2 hidden)
    const void* dh;
    void* dgu;              // (rows, 2 hidden), rows ld apart
    void* dgu_t;            // (2 hidden, rows), rows ld_t apart
    int64_t dh_stride;
    int ld, ld_t;
    int rows, hidden, act;
    unsigned* flags;        // `nflags` arrival counters to clear for a K split that follows
    int nflags;
    GradMask* over;         // F16: every tile's rows (hidden fastest), then its units of dg, then of du
    // launch_gated_repair
    const void* x;
    const void* w;
    void* dx;
    void* dw;
    int64_t x_stride, w_stride;
    int cols;
};
hipError_t launch_gated_grad(const GatedGradArgs& a, int dt, hipStream_t stream);
// F16, behind the products: the rows of dx and dweight that `over` names once more
hipError_t launch_gated_repair(const GatedGradArgs& a, hipStream_t stream);

hipError_t launch_quantize_rows(const void* x, int64_t x_stride, signed char* q, float* scale, int rows,
                                int cols, int dt, hipStream_t stream);

}  // namespace gemm_relu_hip
