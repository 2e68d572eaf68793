// sandwich_norm_f32.cu -- instances of the norms around a block for F32.
#include "sandwich_forward.cuh"

namespace sg {
cudaError_t launch_sandwich_norm_f32(const SandwichParams &p, int sm_count, cudaStream_t s) {
  return launch_norms<float>(p, sm_count, s);
}
}  // namespace sg
