// Instantiations: a dense layer's output tiles, transposed; weight [K,N] MN-major, x K-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear, EPI_LINEAR, true, false, 256)
FLCE_DEFINE_LAUNCHER(launch_linear_128, EPI_LINEAR, true, false, 128)
}  // namespace flce
