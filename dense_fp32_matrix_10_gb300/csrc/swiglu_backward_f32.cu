// swiglu_backward_f32.cu -- instances of the gated unit's gradient for F32.
#include "swiglu_backward.cuh"

namespace sg {
cudaError_t launch_swiglu_backward_f32(const SwigluGradParams &p, int sm_count, cudaStream_t s) {
  return launch_unit_gradient<float>(p, sm_count, s);
}
}  // namespace sg
