// Matrix products of the feed-forward operators: the tile kernel with the gated,
// the plain and the scaled integer epilogue.
#include "ffn.hpp"

namespace gemm_relu_hip {

namespace {

template <class C> __global__ void __launch_bounds__(C::NTHREADS, 1) linear_kernel(KernelArgs args)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[C::LDS_BYTES];
    gemm_relu_tile<C>(args, (int)blockIdx.x, (GR_LDS unsigned char*)(smem_raw), nullptr,
                      Region{args.tiles_m, args.tiles_n, args.panel, 0});
}

template <class C> hipError_t launch(const KernelArgs& args, int grid, hipStream_t stream)
{
    void* params[] = {const_cast<KernelArgs*>(&args)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&linear_kernel<C>), dim3(grid), dim3(C::NTHREADS),
                           params, 0, stream);
}

template <class C> __global__ void __launch_bounds__(C::NTHREADS, 1) linear_pair_kernel(LinearPair pair)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[C::LDS_BYTES];
    const bool second = (int)blockIdx.x >= pair.first;
    const KernelArgs& args = second ? pair.b : pair.a;
    const int wg = (int)blockIdx.x - (second ? pair.first : 0), tiles = args.tiles_m * args.tiles_n;
    // a K split's workgroups take part wg / tiles of tile wg % tiles
    gemm_relu_tile<C>(args, C::SPLITK ? wg % tiles : wg, (GR_LDS unsigned char*)(smem_raw), nullptr,
                      Region{args.tiles_m, args.tiles_n, args.panel, 0, C::SPLITK ? wg / tiles : 0});
}

template <class C> hipError_t launch_pair(const LinearPair& pair, int grid, hipStream_t stream)
{
    void* params[] = {const_cast<LinearPair*>(&pair)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&linear_pair_kernel<C>), dim3(grid), dim3(C::NTHREADS),
                           params, 0, stream);
}

// EPI over inputs IN.  What a configuration measured, in us: 256 x 256, gated 4096 x
// 7168 x 4096 bf16 395 (1.22 PFLOP/s; 128 x 128 485-500) and 8-bit 8192^3 443 (2.48
// POP/s); LIN_128, gated 1024 x 2048 x 1536, one round, 15.4 (LIN_128X2 23, 64 x 64
// 23); LIN_128X2, gated 4096 x 1000 x 1000, 500 tiles, 28 (LIN_128 33, 256 x 256
// 38); 64 x 64, gated 64 x 8192 x 8192 60 (LIN_128 83).  32 x 32 blocks with four
// waves measured 3-15 % slower for LIN_128X2, and 556 us for the 8-bit 8192^3.
//
// Gated and integer products take B stored (N,K) and
// 16x16 blocks everywhere: the two blocks a gated wave needs side by side fit
// the small tiles, and the integer instruction has no other form here.
template <int IN, int OUT, int EPI, int cfg> struct LinearCfg;
template <int IN, int BK16> constexpr int bk = IN == DT_I8 ? 2 * BK16 : BK16;
template <int EPI> constexpr bool nt = EPI != EPI_CAST;
template <int EPI> constexpr int mb = EPI == EPI_CAST ? 32 : 16;

template <int IN, int OUT, int EPI> struct LinearCfg<IN, OUT, EPI, LIN_256> {
    using type = Cfg<IN, OUT, nt<EPI>, 256, 256, bk<IN, 32>, 2, 4, 4, true, true, 16, false, false, false, EPI>;
};
template <int IN, int OUT, int EPI> struct LinearCfg<IN, OUT, EPI, LIN_128> {
    using type = Cfg<IN, OUT, nt<EPI>, 128, 128, bk<IN, 64>, 2, 4, 4, true, true, 16, false, false, false, EPI>;
};
template <int IN, int OUT, int EPI> struct LinearCfg<IN, OUT, EPI, LIN_128X2> {
    using type = Cfg<IN, OUT, nt<EPI>, 128, 128, bk<IN, 64>, 2, 4, 2, true, false, 16, false, false, false, EPI>;
};
template <int IN, int OUT, int EPI> struct LinearCfg<IN, OUT, EPI, LIN_64> {
    using type = Cfg<IN, OUT, nt<EPI>, 64, 64, bk<IN, 64>, 2, 2, 4, true, false, mb<EPI>, false, false, EPI == EPI_CAST, EPI>;
};
template <int IN, int OUT, int EPI> struct LinearCfg<IN, OUT, EPI, LIN_G64> {
    using type = Cfg<IN, OUT, nt<EPI>, 64, 64, bk<IN, 64>, 2, 2, 2, false, false, mb<EPI>, false, false, false, EPI>;
};
template <int IN, int OUT, int EPI> LinearLaunchFn pick(int cfg)
{
    switch (cfg) {
    case LIN_256: return &launch<typename LinearCfg<IN, OUT, EPI, LIN_256>::type>;
    case LIN_128: return &launch<typename LinearCfg<IN, OUT, EPI, LIN_128>::type>;
    case LIN_128X2: return &launch<typename LinearCfg<IN, OUT, EPI, LIN_128X2>::type>;
    case LIN_64: return &launch<typename LinearCfg<IN, OUT, EPI, LIN_64>::type>;
    case LIN_G64: return &launch<typename LinearCfg<IN, OUT, EPI, LIN_G64>::type>;
    default: return nullptr;
    }
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
