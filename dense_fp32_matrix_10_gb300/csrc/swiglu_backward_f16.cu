// swiglu_backward_f16.cu -- instances of the gated unit's gradient for F16.
#include "swiglu_backward.cuh"

namespace sg {
cudaError_t launch_swiglu_backward_f16(const SwigluGradParams &p, int sm_count, cudaStream_t s) {
  return launch_unit_gradient<__half>(p, sm_count, s);
}
}  // namespace sg
