// sandwich_norm_f16.cu -- instances of the norms around a block for F16.
#include "sandwich_forward.cuh"

namespace sg {
cudaError_t launch_sandwich_norm_f16(const SandwichParams &p, int sm_count, cudaStream_t s) {
  return launch_norms<__half>(p, sm_count, s);
}
}  // namespace sg
