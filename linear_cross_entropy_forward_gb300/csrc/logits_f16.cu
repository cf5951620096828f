// Instantiations: kernels of the processed logits for logits of fp16.
#include "flce_logits.cuh"

namespace flce {
namespace logits {
int run_f16(const Args& a, int count, int mode, int sms, cudaStream_t st) {
  return run_type<__half>(a, count, mode, sms, st);
}
}  // namespace logits
}  // namespace flce
