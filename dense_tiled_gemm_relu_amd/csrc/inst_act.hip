// Products with bias, activation and residual in the tile kernel's epilogue, and both
// products of their gradient with the bias's.
#include "linear_tiles.hpp"

namespace gemm_relu_hip {

namespace {

// 64 columns' sums over the strips, in order: each wave takes every NWAVES-th strip, in
// batches of 8 whose loads are in flight together (strips past the end are the last one's,
// and count for nothing).  As a launch of its own it took 4.5 us, whatever its size.
template <int WAVES> __device__ __forceinline__ void sum_strips(const LinearSums& a, int block, GR_LDS float* part)
{
    const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
    const int64_t j = (int64_t)block * 64 + lane;
    float s = 0.0f;
    if (j < a.cols)
        for (int k = wave; k < a.strips; k += WAVES * 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = a.partial[(size_t)min(k + WAVES * u, a.strips - 1) * (size_t)a.cols + j];
#pragma unroll
            for (int u = 0; u < 8; ++u) s += k + WAVES * u < a.strips ? v[u] : 0.0f;
        }
    part[wave * 64 + lane] = s;
    __syncthreads();
    if (wave || j >= a.cols) return;
#pragma unroll
    for (int k = 1; k < WAVES; ++k) s += part[k * 64 + lane];
    if (a.out_dt == DT_F32)
        static_cast<float*>(a.out)[j] = s;
    else if (a.out_dt == DT_F16)
        static_cast<_Float16*>(a.out)[j] = (_Float16)s;
    else
        static_cast<__bf16*>(a.out)[j] = (__bf16)s;
}

template <class C> __global__ void __launch_bounds__(C::NTHREADS, 1) linear_pair_sums_kernel(LinearPairSums p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[C::LDS_BYTES];
    if ((int)blockIdx.x < p.products)
        pair_tile<C>(p.pair, (GR_LDS unsigned char*)(smem_raw));
    else
        sum_strips<C::NWAVES>(p.sums, (int)blockIdx.x - p.products, (GR_LDS float*)(smem_raw));
}
template <class C> hipError_t launch_pair_sums(const LinearPairSums& p, int grid, hipStream_t stream)
{
    void* params[] = {const_cast<LinearPairSums*>(&p)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&linear_pair_sums_kernel<C>), dim3(grid), dim3(C::NTHREADS), params, 0,
                           stream);
}
template <int DT> PairSumsLaunchFn pick_pair_sums(int cfg)
{
    switch (cfg) {
    case LIN_256: return &launch_pair_sums<typename LinearCfg<DT, DT, EPI_CAST, LIN_256>::type>;
    case LIN_128: return &launch_pair_sums<typename LinearCfg<DT, DT, EPI_CAST, LIN_128>::type>;
    case LIN_128X2: return &launch_pair_sums<typename LinearCfg<DT, DT, EPI_CAST, LIN_128X2>::type>;
    case LIN_64: return &launch_pair_sums<typename LinearCfg<DT, DT, EPI_CAST, LIN_64>::type>;
    case LIN_G64: return &launch_pair_sums<typename LinearCfg<DT, DT, EPI_CAST, LIN_G64>::type>;
    default: return nullptr;
    }
}

}  // namespace

LinearLaunchFn launcher_act(int dt, int cfg)
{
    if (cfg >= LIN_K16) return launcher_skinny_act(dt, cfg);
    if (dt == DT_F16) return pick<DT_F16, DT_F16, EPI_ACT>(cfg);
    if (dt == DT_BF16) return pick<DT_BF16, DT_BF16, EPI_ACT>(cfg);
    return nullptr;
}

PairSumsLaunchFn launcher_cast_pair_sums(int dt, int cfg)
{
    if (dt == DT_F16) return pick_pair_sums<DT_F16>(cfg);
    if (dt == DT_BF16) return pick_pair_sums<DT_BF16>(cfg);
    return nullptr;
}

}  // namespace gemm_relu_hip
