// Instantiation: a dense layer's output tiles; x K-major, weight [K,N] MN-major.
#include "flce_gemm.cuh"

namespace flce {
FLCE_DEFINE_LAUNCHER(launch_linear, EPI_LINEAR, false, true, 256)
}  // namespace flce
