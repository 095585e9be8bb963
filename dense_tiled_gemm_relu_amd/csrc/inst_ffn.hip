// Matrix products of the feed-forward operators: the tile kernel with the gated,
// the plain and the scaled integer epilogue.
#include "ffn.hpp"

namespace gemm_relu_hip {

namespace {

template <class C> __global__ void __launch_bounds__(C::NTHREADS, 1) linear_kernel(KernelArgs args)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[C::LDS_BYTES];
    gemm_relu_tile<C>(args, blockIdx.x, (GR_LDS unsigned char*)(smem_raw), nullptr,
                      Region{args.tiles_m, args.tiles_n, args.panel, 0});
}

template <class C> hipError_t launch(const KernelArgs& args, int grid, hipStream_t stream)
{
    void* params[] = {const_cast<KernelArgs*>(&args)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&linear_kernel<C>), dim3(grid), dim3(C::NTHREADS),
                           params, 0, stream);
}

// EPI over inputs IN: gated and integer products take B stored (N,K)
template <int IN, int OUT, int EPI, int cfg> struct LinearCfg;
template <int IN, int OUT, int EPI> struct LinearCfg<IN, OUT, EPI, LIN_G64> {
    static constexpr int BK = IN == DT_I8 ? 128 : 64, MB = EPI == EPI_CAST ? 32 : 16;
    using type = Cfg<IN, OUT, EPI != EPI_CAST, 64, 64, BK, 2, 2, 2, false, false, MB, false, false, false, EPI>;
};

template <int IN, int OUT, int EPI> LinearLaunchFn pick(int cfg)
{
    switch (cfg) {
    case LIN_G64: return &launch<typename LinearCfg<IN, OUT, EPI, LIN_G64>::type>;
    default: return nullptr;
    }
}

}  // namespace

LinearLaunchFn launcher_gated(int dt, int cfg)
{
    if (dt == DT_F16) return pick<DT_F16, DT_F16, EPI_GATED>(cfg);
    if (dt == DT_BF16) return pick<DT_BF16, DT_BF16, EPI_GATED>(cfg);
    return nullptr;
}

LinearLaunchFn launcher_cast(int dt, int cfg)
{
    if (dt == DT_F16) return pick<DT_F16, DT_F16, EPI_CAST>(cfg);
    if (dt == DT_BF16) return pick<DT_BF16, DT_BF16, EPI_CAST>(cfg);
    return nullptr;
}

LinearLaunchFn launcher_i8(int out_dt, int cfg)
{
    if (out_dt == DT_F16) return pick<DT_I8, DT_F16, EPI_I8>(cfg);
    if (out_dt == DT_BF16) return pick<DT_I8, DT_BF16, EPI_I8>(cfg);
    if (out_dt == DT_F32) return pick<DT_I8, DT_F32, EPI_I8>(cfg);
    return nullptr;
}

}  // namespace gemm_relu_hip
