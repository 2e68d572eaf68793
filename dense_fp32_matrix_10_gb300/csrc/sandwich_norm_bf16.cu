// sandwich_norm_bf16.cu -- instances of the norms around a block for BF16.
#include "sandwich_forward.cuh"

namespace sg {
cudaError_t launch_sandwich_norm_bf16(const SandwichParams &p, int sm_count, cudaStream_t s) {
  return launch_norms<__nv_bfloat16>(p, sm_count, s);
}
}  // namespace sg
