// swiglu.cuh -- the logistic function of the gated unit's kernels.
#pragma once

#include "fp8_block.cuh"

namespace sg {

// -1 / (1 + exp(-g)); 0 where the exponential leaves FP32.
__device__ __forceinline__ float negated_logistic(float g) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  return rcp_approx(-1.0f - e);
}
__device__ __forceinline__ float2 negated_logistic(float2 g) {
  return make_float2(negated_logistic(g.x), negated_logistic(g.y));
}

}  // namespace sg
