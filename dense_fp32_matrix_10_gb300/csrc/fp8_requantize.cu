// fp8_requantize.cu -- from 1 x 128 to 128 x 1 blocks: x = q s, and per column
// of 128 rows s' = max(max|x| / F, 2^-126), q' = fp8(x / s').
//
// One CTA takes a 128 x 128 tile, 16 lanes a row: the 8-bit elements stay in
// registers between the maxima and the quotients.
#include "dispatch.h"
#include "fp8_block.cuh"

namespace sg {
namespace {

__global__ void __launch_bounds__(256) requantize_kernel(const RequantizeParams p, const int64_t tiles_c, const bool vec_x,
                                                         const bool vec_q) {
  __shared__ float part[8][128];   // column maxima of each warp, then -1 / scale and scale of the tile
  griddep_wait();
  griddep_launch_dependents();
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t c = tc * 128 + lane16 * 8, r0 = tr * 128 + row16;   // this thread's rows: r0 + 16 i
  const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c)));
  const int rows = static_cast<int>(min(int64_t(128), p.rows - r0));
  uint2 raw[8];
  float sx[8], cmax[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    raw[i] = load8_fp8(p.x + (r0 + 16 * i) * p.ldx + c, 16 * i < rows ? n : 0, vec_x);
    sx[i] = 16 * i < rows ? p.sx[(r0 + 16 * i) * p.ldsx + tc] : 0.0f;
    cmax[i] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack_fp8(raw[i], p.x_e5m2, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = max_abs(cmax[j], v[j] * sx[i]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cmax[j] = max_abs(cmax[j], __shfl_xor_sync(~0u, cmax[j], 16));
    if ((threadIdx.x & 16) == 0) part[warp][lane16 * 8 + j] = cmax[j];
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    float a = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) a = max_abs(a, part[w][threadIdx.x]);
    const float s = block_scale(a, p.e5m2);
    const int64_t at = tc * 128 + threadIdx.x;
    if (at < p.cols) p.s[tr * p.lds + at] = s;
    part[0][threadIdx.x] = __fdiv_rn(-1.0f, s);
    part[1][threadIdx.x] = divisor(s);
  }
  __syncthreads();
  float ninv[8], div[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    ninv[j] = part[0][lane16 * 8 + j];
    div[j] = part[1][lane16 * 8 + j];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack_fp8(raw[i], p.x_e5m2, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = quotient(v[j] * sx[i], div[j], ninv[j]);
    if (16 * i < rows) store8_fp8(p.q + (r0 + 16 * i) * p.ldq + c, to_fp8x8(v, 1.0f, p.e5m2), n, vec_q);
  }
}

}  // namespace

cudaError_t launch_requantize(const RequantizeParams &p, cudaStream_t s) {
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = tiles_c * ((p.rows + 127) / 128);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_maybe_pdl(requantize_kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, true, p, tiles_c,
                          aligned_rows(p.x, p.ldx, 1, 8), aligned_rows(p.q, p.ldq, 1, 8));
}

}  // namespace sg
