// fp8_quantize.cu -- quantisation in blocks of 1 x 128, 128 x 1 (or both at
// once) and 128 x 128: s = max(max|x| / F, 2^-126), q = fp8(x / s).
//
// One CTA takes a 128 x 128 tile, so that every block of any of the forms lies
// in one CTA: x is read once, held in registers in its own type, and the
// maxima go over 16 lanes (rows) and over the tile's row groups through
// shared memory (columns).  Bound by memory: T + 1 bytes an element (T + 2
// for both).
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace sg {
namespace {

enum : int { kRow = 1, kCol = 2, kTile = 4 };

template <class T, int MODE>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantizeParams p, const int64_t tiles_c,
                                                       const bool vec_x, const bool vec_r,
                                                       const bool vec_c) {
  __shared__ float part[8][128];   // column maxima of each warp, then of the tile
  griddep_wait();
  griddep_launch_dependents();
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t c0 = tc * 128 + lane16 * 8;
  const int64_t left = p.cols - c0;
  const int n = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
  Raw<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = tr * 128 + row16 + 16 * i;
    raw[i] = load8(static_cast<const T *>(p.x) + (r < p.rows ? r * p.ldx + c0 : 0), r < p.rows ? n : 0, vec_x);
  }
  float cmax[8], tmax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack(raw[i], v);
    if (MODE & kCol) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax[j] = max_abs(cmax[j], v[j]);
    }
    if (MODE & (kRow | kTile)) {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = max_abs(a, v[j]);
      if (MODE & kTile) {
        tmax = max_abs(tmax, a);
      } else {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) a = max_abs(a, __shfl_xor_sync(~0u, a, d));
        const float s = block_scale(a, p.e5m2);
        const int64_t r = tr * 128 + row16 + 16 * i;
        if (r < p.rows) {
          store8_fp8(p.qr + r * p.ldqr + c0, to_fp8x8(v, __fdiv_rn(1.0f, s), p.e5m2), n, vec_r);
          if (lane16 == 0) p.sr[r * p.ldsr + tc] = s;
        }
      }
    }
  }
  if (MODE & kTile) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) tmax = max_abs(tmax, __shfl_xor_sync(~0u, tmax, d));
    if ((threadIdx.x & 31) == 0) part[0][warp] = tmax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) tmax = max_abs(tmax, part[0][w]);
    const float s = block_scale(tmax, p.e5m2), inv = __fdiv_rn(1.0f, s);
    if (threadIdx.x == 0) p.sr[tr * p.ldsr + tc] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = tr * 128 + row16 + 16 * i;
      float v[8];
      unpack(raw[i], v);
      if (r < p.rows) store8_fp8(p.qr + r * p.ldqr + c0, to_fp8x8(v, inv, p.e5m2), n, vec_r);
    }
  }
  if (MODE & kCol) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = max_abs(cmax[j], __shfl_xor_sync(~0u, cmax[j], 16));
    if ((threadIdx.x & 31) < 16) {
#pragma unroll
      for (int j = 0; j < 8; ++j) part[warp][lane16 * 8 + j] = cmax[j];
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      float a = part[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) a = max_abs(a, part[w][threadIdx.x]);
      const float s = block_scale(a, p.e5m2);
      const int64_t c = tc * 128 + threadIdx.x;
      if (c < p.cols) p.sc[tr * p.ldsc + c] = s;
      part[0][threadIdx.x] = __fdiv_rn(1.0f, s);
    }
    __syncthreads();
    float inv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = part[0][lane16 * 8 + j];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = tr * 128 + row16 + 16 * i;
      float v[8];
      unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= inv[j];
      if (r < p.rows) store8_fp8(p.qc + r * p.ldqc + c0, to_fp8x8(v, 1.0f, p.e5m2), n, vec_c);
    }
  }
}

template <class T>
cudaError_t launch_typed(const QuantizeParams &p, cudaStream_t s) {
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = tiles_c * ((p.rows + 127) / 128);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const bool vx = aligned_rows(p.x, p.ldx, sizeof(T), 16);
  const bool vr = p.qr && aligned_rows(p.qr, p.ldqr, 1, 8), vc = p.qc && aligned_rows(p.qc, p.ldqc, 1, 8);
  const dim3 grid(static_cast<unsigned>(tiles)), block(256);
  auto go = [&](auto kernel) { return launch_maybe_pdl(kernel, grid, block, 0, s, true, p, tiles_c, vx, vr, vc); };
  if (p.tile) return go(quantize_kernel<T, kTile>);
  if (p.qr && p.qc) return go(quantize_kernel<T, kRow | kCol>);
  return p.qr ? go(quantize_kernel<T, kRow>) : go(quantize_kernel<T, kCol>);
}

}  // namespace

cudaError_t launch_quantize(const QuantizeParams &p, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return launch_typed<float>(p, s);
    case SGEMM_TYPE_BF16: return launch_typed<__nv_bfloat16>(p, s);
    default: return launch_typed<__half>(p, s);
  }
}

}  // namespace sg
