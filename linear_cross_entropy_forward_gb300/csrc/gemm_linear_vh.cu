// Instantiation: a dense layer's output tiles; x K-major, weight [N,K] K-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear_vh, EPI_LINEAR, false, false, 256)
}  // namespace flce
