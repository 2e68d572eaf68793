// fp8.h -- parameters and launchers of the 8-bit linear layer's kernels (host
// side).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sgemm_fp8.h"

namespace sg {

// One 8-bit operand of a product.
struct Fp8Operand {
  const unsigned char *q;
  const float *s;
  int64_t ld, lds;
  int e5m2;        // element type: E5M2 rather than E4M3
  int inner_rows;  // the inner dimension k runs along the rows of the stored matrix (its columns
                   // are the outer dimension); otherwise k is contiguous
  int shift;       // outer index >> shift = index of its scale (0 or 7)
};

struct Fp8Params {
  Fp8Operand a, b;
  void *C;
  int64_t ldc;
  int M, N, K;
  int typeC;   // sgemm_type_t
  float alpha, beta;
  uint64_t wait_budget_ns;
  int *status;
};

// The form of the kernel for a product, and the CTAs that share a tile's blocks of k (fp8_tc.cu).
struct Fp8Choice {
  sgemm_fp8_form_t form;
  int split;
};
Fp8Choice choose_fp8_form(const Fp8Params &p, int sm_count);
// The product on the tensor cores, any layout (fp8_tc.cu).
cudaError_t launch_fp8_product(const Fp8Params &p, int sm_count, cudaStream_t s);
// C = beta * C (fp8_scale_c.cu).
cudaError_t launch_fp8_scale_c(const Fp8Params &p, cudaStream_t s);

struct QuantizeParams {
  const void *x;
  int64_t ldx, rows, cols;
  int typeX, e5m2;
  unsigned char *qr, *qc;   // 1 x 128 (or 128 x 128) and 128 x 1 outputs
  float *sr, *sc;
  int64_t ldqr, ldqc, ldsr, ldsc;
  int tile;                 // qr, sr hold 128 x 128 blocks
};
cudaError_t launch_quantize(const QuantizeParams &p, cudaStream_t s);

struct NormParams {
  const void *x, *r, *w;
  void *h, *y;
  unsigned char *q;
  float *s, *t;
  int64_t ldx, ldr, ldh, ldy, ldq, lds, rows, cols;
  int typeX, w_f32, e5m2;
  float eps;
};
cudaError_t launch_rms_norm(const NormParams &p, int sm_count, cudaStream_t s);

// CTAs of the backward kernel, each with a partial sum of dw, at most (for any type).
int64_t norm_partials(int64_t rows, int64_t cols);
struct NormGradParams {
  const void *dy, *h, *w, *dh;
  const float *t;
  void *dx, *dw;
  float *partial;   // one row of ceil(cols / 8) * 8 floats per CTA
  int64_t lddy, ldh, lddh, lddx, rows, cols;
  int typeX, w_f32;
};
cudaError_t launch_rms_norm_backward(const NormGradParams &p, cudaStream_t s);

}  // namespace sg
