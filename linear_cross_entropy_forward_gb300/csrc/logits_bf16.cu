// Instantiations: kernels of the processed logits for logits of bf16.
#include "flce_logits.cuh"

namespace flce {
namespace logits {
int run_bf16(const Args& a, int count, int mode, int sms, cudaStream_t st) {
  return run_type<__nv_bfloat16>(a, count, mode, sms, st);
}
}  // namespace logits
}  // namespace flce
