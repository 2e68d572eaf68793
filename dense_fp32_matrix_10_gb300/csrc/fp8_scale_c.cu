// fp8_scale_c.cu -- what is left of the 8-bit product when there is nothing to multiply: C = beta * C (zeros
// without reading C when beta is 0).
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace sg {
namespace {

template <class T>
__global__ void __launch_bounds__(256) fp8_scale_c_kernel(const Fp8Params p) {
  griddep_wait();
  const int64_t total = static_cast<int64_t>(p.M) * p.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    T *c = static_cast<T *>(p.C) + i / p.N * p.ldc + i % p.N;
    from_float(c, p.beta != 0.0f ? p.beta * to_float(*c) : 0.0f);
  }
}

}  // namespace

cudaError_t launch_fp8_scale_c(const Fp8Params &p, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(p.M) * p.N + 1023) / 1024;
  const dim3 grid(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), block(256);
  switch (p.typeC) {
    case SGEMM_TYPE_F32: return launch_maybe_pdl(fp8_scale_c_kernel<float>, grid, block, 0, s, true, p);
    case SGEMM_TYPE_BF16: return launch_maybe_pdl(fp8_scale_c_kernel<__nv_bfloat16>, grid, block, 0, s, true, p);
    default: return launch_maybe_pdl(fp8_scale_c_kernel<__half>, grid, block, 0, s, true, p);
  }
}

}  // namespace sg
