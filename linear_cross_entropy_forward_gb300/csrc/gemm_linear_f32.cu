// Instantiations: a dense layer's output tiles in fp32, transposed; weight [K,N] MN-major or [N,K]
// K-major, x K-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear_f32, EPI_LINEAR_F32, true, false, 256)
FLCE_DEFINE_LAUNCHER(launch_linear_vh_f32, EPI_LINEAR_F32, false, false, 256)
}  // namespace flce
