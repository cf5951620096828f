// Instantiations: a dense layer's gradients on tiles of 128 columns (on 256 they are the head's).
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear_dx_128, EPI_ACCUM, false, false, 128)
FLCE_DEFINE_LAUNCHER(launch_linear_dx_vh_128, EPI_ACCUM, false, true, 128)
FLCE_DEFINE_LAUNCHER(launch_linear_dweight_128, EPI_STORE_BF16, true, true, 128)
}  // namespace flce
