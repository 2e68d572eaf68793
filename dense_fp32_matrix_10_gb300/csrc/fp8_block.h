// fp8_block.h -- parameters and launchers of the kernels around a gated
// block's products (host side).  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sgemm_fp8_block.h"

namespace sg {

// A matrix of a call's float type (s null), or its checkpoint.
struct Kept {
  const void *p;
  const float *s;
  int64_t ld, lds;
  int e5m2;
};

// One row for every `rows` consecutive ones (p null: the gate is 1).
struct Gate {
  const void *p;
  int64_t ld;
  unsigned rows;   // at most kMaxDim
  int f32;
};

struct SandwichParams {
  const void *a, *x, *wp, *w;
  Gate gate;
  void *h;
  unsigned char *q, *qa, *qh;
  float *s, *sa, *sh, *tp, *t;
  int64_t lda, ldx, ldh, ldq, lds, ldqa, ldsa, ldqh, ldsh, rows, cols;
  int w_f32, e5m2, keep_e5m2;
  float eps, residual_scale;
};
// (one for each type of a)
cudaError_t launch_sandwich_norm_f32(const SandwichParams &p, int sm_count, cudaStream_t s);
cudaError_t launch_sandwich_norm_bf16(const SandwichParams &p, int sm_count, cudaStream_t s);
cudaError_t launch_sandwich_norm_f16(const SandwichParams &p, int sm_count, cudaStream_t s);

struct SandwichGradParams {
  const void *dy, *dh, *wp, *w;
  Kept a, h;
  Gate gate;
  const float *tp, *t;
  void *da, *dx, *dwp, *dw, *dgate;
  float *partial;
  int64_t lddy, lddh, ldda, lddx, lddgate, rows, cols;
  int typeX, w_f32;
  float residual_scale;
  uint64_t wait_budget_ns;
  int *status;
};
// Floats of workspace.
int64_t sandwich_partials(int64_t rows, int64_t cols);
// *launches: kernels queued.
cudaError_t launch_sandwich_norm_backward(const SandwichGradParams &p, cudaStream_t s, int *launches);

struct SwigluParams {
  const void *g, *u;
  unsigned char *q, *qg, *qu;
  float *s, *sg, *su;
  int64_t ldg, ldu, ldq, lds, ldqg, ldsg, ldqu, ldsu, rows, cols;
  int typeX, e5m2, keep_e5m2;
};
cudaError_t launch_swiglu(const SwigluParams &p, cudaStream_t s);

struct SwigluGradParams {
  const void *dy;
  Kept g, u;
  unsigned char *qr, *qc, *qy;
  float *sr, *sc, *sy;
  int64_t lddy, ldqr, ldsr, ldqc, ldsc, ldqy, ldsy, rows, cols;
  int z_e5m2, y_e5m2;
};
// (one for each type of dy)
cudaError_t launch_swiglu_backward_f32(const SwigluGradParams &p, int sm_count, cudaStream_t s);
cudaError_t launch_swiglu_backward_bf16(const SwigluGradParams &p, int sm_count, cudaStream_t s);
cudaError_t launch_swiglu_backward_f16(const SwigluGradParams &p, int sm_count, cudaStream_t s);

struct RequantizeParams {
  const unsigned char *x;
  const float *sx;
  unsigned char *q;
  float *s;
  int64_t ldx, ldsx, ldq, lds, rows, cols;
  int x_e5m2, e5m2;
};
cudaError_t launch_requantize(const RequantizeParams &p, cudaStream_t s);

}  // namespace sg
