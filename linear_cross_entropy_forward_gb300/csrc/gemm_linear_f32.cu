// Instantiations: a dense layer's output tiles in fp32; x K-major, weight [K,N] MN-major or [N,K] K-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear_f32, EPI_LINEAR_F32, false, true, 256)
FLCE_DEFINE_LAUNCHER(launch_linear_vh_f32, EPI_LINEAR_F32, false, false, 256)
}  // namespace flce
