// swiglu.cu -- the gated unit y = g p u, p = 1 / (1 + exp(-g)), with a
// quantised output, and its gradient as operands of the products that follow:
//
//   du = dy g p,   dg = dy u p (1 + g (1 - p))
//
// The forward pass works on 1 x 128 blocks, 16 lanes a block.  The gradient
// takes 128 x 128 tiles, so that every block of either orientation lies in one
// CTA: 16 lanes a row again, and the column maxima go over the rows' threads
// through shared memory.
#include "dispatch.h"
#include "fp8_block.cuh"

namespace sg {
namespace {

// 1 / (1 + exp(-g)); 0 where the exponential leaves FP32.
__device__ __forceinline__ float logistic(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// vec: bit 0 g, 1 u (16-byte rows), 2 q, 3 qg, 4 qu (8-byte rows)
template <class T>
__global__ void __launch_bounds__(256) swiglu_kernel(const SwigluParams p, const int64_t blocks_c, const int64_t units,
                                                     const int vec) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int64_t row = min(unit, units - 1) / blocks_c, block = min(unit, units - 1) - row * blocks_c;
  const int64_t c = block * 128 + (threadIdx.x & 15) * 8;
  const int n = unit < units ? static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c))) : 0;
  float g[8], u[8], y[8];
  unpack(load8(static_cast<const T *>(p.g) + row * p.ldg + c, n, vec & 1), g);
  unpack(load8(static_cast<const T *>(p.u) + row * p.ldu + c, n, vec & 2), u);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = g[i] * logistic(g[i]) * u[i];
  store_block(y, n, p.q + row * p.ldq + c, p.s + row * p.lds + block, p.e5m2, vec & 4);
  if (p.qg) store_block(g, n, p.qg + row * p.ldqg + c, p.sg + row * p.ldsg + block, p.keep_e5m2, vec & 8);
  if (p.qu) store_block(u, n, p.qu + row * p.ldqu + c, p.su + row * p.ldsu + block, p.keep_e5m2, vec & 16);
}

// ------------------------------------------------------------------ gradient
// vec: bit 0 dy, 1 g, 2 u (16-byte rows, 8-byte of checkpoints), 3 qr, 4 qc, 5 qy (8-byte rows)
template <class T, bool KEPT>
__global__ void __launch_bounds__(512) swiglu_backward_kernel(const SwigluGradParams p, const int64_t tiles_c,
                                                              const int vec) {
  extern __shared__ __align__(16) float part[];   // [16 warps][3][128] column maxima, then -1 / scale and scale of the tile
  griddep_wait();
  griddep_launch_dependents();
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c, wide = tiles_c * 128;
  const int lane16 = threadIdx.x & 15, row32 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t c = tc * 128 + lane16 * 8, r0 = tr * 128 + row32;   // this thread's rows: r0 + 32 i
  const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c)));
  const int rows = static_cast<int>(min(int64_t(128), p.rows - r0));
  float v[3][4][8], cmax[3][8];   // dg, du, y
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[k][j] = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = 32 * i < rows ? n : 0;
    const int64_t row = r0 + 32 * i;
    float dy[8], g[8], u[8];
    unpack(load8(static_cast<const T *>(p.dy) + row * p.lddy + c, m, vec & 1), dy);
    if (KEPT) {
      unpack_fp8(load8_fp8(static_cast<const unsigned char *>(p.g.p) + row * p.g.ld + c, m, vec & 2), p.g.e5m2, g);
      unpack_fp8(load8_fp8(static_cast<const unsigned char *>(p.u.p) + row * p.u.ld + c, m, vec & 4), p.u.e5m2, u);
      const float sg = m > 0 ? p.g.s[row * p.g.lds + tc] : 0.0f, su = m > 0 ? p.u.s[row * p.u.lds + tc] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = j < m ? g[j] * sg : 0.0f;
        u[j] = j < m ? u[j] * su : 0.0f;
      }
    } else {
      unpack(load8(static_cast<const T *>(p.g.p) + row * p.g.ld + c, m, vec & 2), g);
      unpack(load8(static_cast<const T *>(p.u.p) + row * p.u.ld + c, m, vec & 4), u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = logistic(g[j]), gs = g[j] * s;
      v[0][i][j] = dy[j] * u[j] * (s + gs * (1.0f - s));
      v[1][i][j] = dy[j] * gs;
      v[2][i][j] = gs * u[j];
#pragma unroll
      for (int k = 0; k < 3; ++k) cmax[k][j] = max_abs(cmax[k][j], v[k][i][j]);
    }
    // the row blocks of dg and du
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = max_abs(a, v[k][i][j]);
      const float s = block_scale(max_of_16(a), p.z_e5m2);
      if (32 * i < rows) {
        store8_fp8(p.qr + row * p.ldqr + k * wide + c, quantize8(v[k][i], divisor(s), __fdiv_rn(-1.0f, s), p.z_e5m2), 8,
                   vec & 8);
        if (lane16 == 0) p.sr[row * p.ldsr + k * tiles_c + tc] = s;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cmax[k][j] = max_abs(cmax[k][j], __shfl_xor_sync(~0u, cmax[k][j], 16));
      if ((threadIdx.x & 16) == 0) part[(warp * 3 + k) * 128 + lane16 * 8 + j] = cmax[k][j];
    }
  __syncthreads();
  float scale = 0.0f;
  const int kind = threadIdx.x >> 7, col = threadIdx.x & 127;   // threads 0 .. 383
  if (threadIdx.x < 384) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) a = max_abs(a, part[(w * 3 + kind) * 128 + col]);
    scale = block_scale(a, kind == 2 ? p.y_e5m2 : p.z_e5m2);
    const int64_t at = tc * 128 + col;
    if (kind < 2)
      p.sc[tr * p.ldsc + kind * wide + at] = scale;
    else if (at < p.cols)
      p.sy[tr * p.ldsy + at] = scale;
  }
  __syncthreads();
  if (threadIdx.x < 384) {
    part[threadIdx.x] = __fdiv_rn(-1.0f, scale);
    part[384 + threadIdx.x] = divisor(scale);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    float ninv[8], div[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ninv[j] = part[k * 128 + lane16 * 8 + j];
      div[j] = part[384 + k * 128 + lane16 * 8 + j];
    }
    unsigned char *q = k < 2 ? p.qc + r0 * p.ldqc + k * wide + c : p.qy + r0 * p.ldqy + c;
    const int64_t ld = k < 2 ? p.ldqc : p.ldqy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = quotient(v[k][i][j], div[j], ninv[j]);
      if (32 * i < rows)
        store8_fp8(q + 32 * i * ld, to_fp8x8(o, 1.0f, k < 2 ? p.z_e5m2 : p.y_e5m2), k < 2 ? 8 : n,
                   k < 2 ? vec & 16 : vec & 32);
    }
  }
}

template <class T>
cudaError_t forward_typed(const SwigluParams &p, cudaStream_t s) {
  const int64_t blocks_c = (p.cols + 127) / 128, units = blocks_c * p.rows, ctas = (units + 15) / 16;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  const int e = sizeof(T);
  const int vec = (aligned_rows(p.g, p.ldg, e, 16) ? 1 : 0) | (aligned_rows(p.u, p.ldu, e, 16) ? 2 : 0) |
                  (aligned_rows(p.q, p.ldq, 1, 8) ? 4 : 0) | (aligned_rows(p.qg, p.ldqg, 1, 8) ? 8 : 0) |
                  (aligned_rows(p.qu, p.ldqu, 1, 8) ? 16 : 0);
  return launch_maybe_pdl(swiglu_kernel<T>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, true, p, blocks_c, units,
                          vec);
}

template <class T, bool KEPT>
cudaError_t backward_typed(const SwigluGradParams &p, cudaStream_t s) {
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = tiles_c * ((p.rows + 127) / 128);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const int e = sizeof(T), ek = KEPT ? 1 : e, ak = KEPT ? 8 : 16;
  const int vec = (aligned_rows(p.dy, p.lddy, e, 16) ? 1 : 0) | (aligned_rows(p.g.p, p.g.ld, ek, ak) ? 2 : 0) |
                  (aligned_rows(p.u.p, p.u.ld, ek, ak) ? 4 : 0) | (aligned_rows(p.qr, p.ldqr, 1, 8) ? 8 : 0) |
                  (aligned_rows(p.qc, p.ldqc, 1, 8) ? 16 : 0) | (aligned_rows(p.qy, p.ldqy, 1, 8) ? 32 : 0);
  return launch_maybe_pdl(swiglu_backward_kernel<T, KEPT>, dim3(static_cast<unsigned>(tiles)), dim3(512),
                          16 * 3 * 128 * sizeof(float), s, true, p, tiles_c, vec);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluParams &p, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return forward_typed<float>(p, s);
    case SGEMM_TYPE_BF16: return forward_typed<__nv_bfloat16>(p, s);
    default: return forward_typed<__half>(p, s);
  }
}

cudaError_t launch_swiglu_backward(const SwigluGradParams &p, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return p.g.s ? backward_typed<float, true>(p, s) : backward_typed<float, false>(p, s);
    case SGEMM_TYPE_BF16:
      return p.g.s ? backward_typed<__nv_bfloat16, true>(p, s) : backward_typed<__nv_bfloat16, false>(p, s);
    default: return p.g.s ? backward_typed<__half, true>(p, s) : backward_typed<__half, false>(p, s);
  }
}

}  // namespace sg
