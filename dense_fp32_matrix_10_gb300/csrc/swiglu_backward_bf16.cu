// swiglu_backward_bf16.cu -- instances of the gated unit's gradient for BF16.
#include "swiglu_backward.cuh"

namespace sg {
cudaError_t launch_swiglu_backward_bf16(const SwigluGradParams &p, int sm_count, cudaStream_t s) {
  return launch_unit_gradient<__nv_bfloat16>(p, sm_count, s);
}
}  // namespace sg
