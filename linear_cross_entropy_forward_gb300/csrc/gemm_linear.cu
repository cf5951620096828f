// Instantiations: a dense layer's output tiles; x K-major, weight [K,N] MN-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear, EPI_LINEAR, false, true, 256)
FLCE_DEFINE_LAUNCHER(launch_linear_128, EPI_LINEAR, false, true, 128)
}  // namespace flce
