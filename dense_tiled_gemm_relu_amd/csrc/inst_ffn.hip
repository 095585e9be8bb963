// Matrix products of the feed-forward operators: the tile kernel with the gated,
// the plain and the scaled integer epilogue.
#include "linear_tiles.hpp"

namespace gemm_relu_hip {

namespace {

template <class C> __global__ void __launch_bounds__(C::NTHREADS, 1) linear_pair_kernel(LinearPair pair)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[C::LDS_BYTES];
    pair_tile<C>(pair, (GR_LDS unsigned char*)(smem_raw));
}

template <class C> hipError_t launch_pair(const LinearPair& pair, int grid, hipStream_t stream)
{
    void* params[] = {const_cast<LinearPair*>(&pair)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&linear_pair_kernel<C>), dim3(grid), dim3(C::NTHREADS),
                           params, 0, stream);
}

template <int DT> PairLaunchFn pick_pair(int cfg)
{
    switch (cfg) {
    case LIN_256: return &launch_pair<typename LinearCfg<DT, DT, EPI_CAST, LIN_256>::type>;
    case LIN_128: return &launch_pair<typename LinearCfg<DT, DT, EPI_CAST, LIN_128>::type>;
    case LIN_128X2: return &launch_pair<typename LinearCfg<DT, DT, EPI_CAST, LIN_128X2>::type>;
    case LIN_64: return &launch_pair<typename LinearCfg<DT, DT, EPI_CAST, LIN_64>::type>;
    case LIN_G64: return &launch_pair<typename LinearCfg<DT, DT, EPI_CAST, LIN_G64>::type>;
    default: return nullptr;
    }
}

}  // namespace

LinearLaunchFn launcher_gated(int dt, int cfg)
{
    if (cfg >= LIN_K16) return launcher_skinny_gated(dt, cfg);
    if (dt == DT_F16) return pick<DT_F16, DT_F16, EPI_GATED>(cfg);
    if (dt == DT_BF16) return pick<DT_BF16, DT_BF16, EPI_GATED>(cfg);
    return nullptr;
}

PairLaunchFn launcher_cast_pair(int dt, int cfg)
{
    if (dt == DT_F16) return pick_pair<DT_F16>(cfg);
    if (dt == DT_BF16) return pick_pair<DT_BF16>(cfg);
    return nullptr;
}

LinearLaunchFn launcher_i8(int out_dt, int cfg)
{
    if (cfg >= LIN_K16) return launcher_skinny_i8(out_dt, cfg);
    if (out_dt == DT_F16) return pick<DT_I8, DT_F16, EPI_I8>(cfg);
    if (out_dt == DT_BF16) return pick<DT_I8, DT_BF16, EPI_I8>(cfg);
    if (out_dt == DT_F32) return pick<DT_I8, DT_F32, EPI_I8>(cfg);
    return nullptr;
}

}  // namespace gemm_relu_hip
