// Products with bias, activation and residual in the tile kernel's epilogue.
#include "linear_tiles.hpp"

namespace gemm_relu_hip {

LinearLaunchFn launcher_act(int dt, int cfg)
{
    if (cfg >= LIN_K16) return launcher_skinny_act(dt, cfg);
    if (dt == DT_F16) return pick<DT_F16, DT_F16, EPI_ACT>(cfg);
    if (dt == DT_BF16) return pick<DT_BF16, DT_BF16, EPI_ACT>(cfg);
    return nullptr;
}

}  // namespace gemm_relu_hip
