// Instantiations: a dense layer's output tiles, transposed; weight [N,K] and x both K-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear_vh, EPI_LINEAR, false, false, 256)
FLCE_DEFINE_LAUNCHER(launch_linear_vh_128, EPI_LINEAR, false, false, 128)
}  // namespace flce
