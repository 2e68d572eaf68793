// fp8_requantize.cu -- from 1 x 128 to 128 x 1 blocks: x = q s, and per column
// of 128 rows s' = max(max|x| / F, 2^-126), q' = fp8(x / s').
//
// One CTA takes a 128 x 128 tile, eight lanes a row and 16 elements a lane:
// the 8-bit elements stay in registers between the maxima and the quotients.
// 12 instructions an element, 69 % of the issue slots: 8192 x 8192 34 us, 4.1
// TB/s, 16384 x 8192 63 us.
#include "dispatch.h"
#include "fp8_block.cuh"

namespace sg {
namespace {

template <bool XE5M2, bool E5M2>
__global__ void __launch_bounds__(256, 4) requantize_kernel(const RequantizeParams p, const unsigned tiles_c, const uint32_t vec) {
  __shared__ __align__(16) float part[8][128];   // column maxima of each warp
  __shared__ __align__(16) float inv[2][128];    // the columns' -1 / scale and scale, at column_place()
  griddep_wait();
  griddep_launch_dependents();
  const unsigned tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int lane8 = threadIdx.x & 7, row32 = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(tc) * 128 + lane8 * 16;
  const int64_t r0 = static_cast<int64_t>(tr) * 128 + row32;   // this thread's rows: r0 + 32 i
  const int n = static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - c)));
  const int rows = static_cast<int>(min(int64_t(128), p.rows - r0));
  uint4 raw[4];
  float sx[4];
  {
    const unsigned char *x = p.x + r0 * p.ldx + c;
    const float *s = p.sx + r0 * p.ldsx + tc;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw[i] = load16_fp8(x + 32 * i * p.ldx, 32 * i < rows ? n : 0, level(vec, 0));
      sx[i] = 32 * i < rows ? s[32 * i * p.ldsx] : 0.0f;
    }
  }
  float2 cmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[j] = both(0.0f);
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    float2 v[8], w[8];
    unpack_fp8<XE5M2>(raw[i], v);
    unpack_fp8<XE5M2>(raw[i + 1], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = mul2(v[j], both(sx[i]));
      w[j] = mul2(w[j], both(sx[i + 1]));
      cmax[j] = make_float2(max_abs3(cmax[j].x, v[j].x, w[j].x), max_abs3(cmax[j].y, v[j].y, w[j].y));
    }
  }
  // over the warp's four rows: a lane keeps the half of its columns that it owns, then half of those
  {
    const bool h16 = threadIdx.x & 16, h8 = threadIdx.x & 8;
    float2 a[4], b[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 mine = h16 ? cmax[4 + j] : cmax[j], give = h16 ? cmax[j] : cmax[4 + j];
      a[j] = make_float2(max_abs(mine.x, __shfl_xor_sync(~0u, give.x, 16)), max_abs(mine.y, __shfl_xor_sync(~0u, give.y, 16)));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 mine = h8 ? a[2 + j] : a[j], give = h8 ? a[j] : a[2 + j];
      b[j] = make_float2(max_abs(mine.x, __shfl_xor_sync(~0u, give.x, 8)), max_abs(mine.y, __shfl_xor_sync(~0u, give.y, 8)));
    }
    *reinterpret_cast<float4 *>(&part[warp][lane8 * 16 + (h16 ? 8 : 0) + (h8 ? 4 : 0)]) =
        make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    float a = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 7; w += 2) a = max_abs3(a, part[w][threadIdx.x], part[w + 1][threadIdx.x]);
    a = max_abs(a, part[7][threadIdx.x]);
    const float s = scale_of(a, E5M2);
    const int64_t at = static_cast<int64_t>(tc) * 128 + threadIdx.x;
    if (at < p.cols) p.s[tr * p.lds + at] = s;
    inv[0][column_place(threadIdx.x)] = ninv_of(s);
    inv[1][column_place(threadIdx.x)] = divisor(s);
  }
  __syncthreads();
  // (without this the compiler keeps the 64 unpacked values of the maxima, in registers that the kernel does not have)
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("" : "+r"(raw[i].x), "+r"(raw[i].y), "+r"(raw[i].z), "+r"(raw[i].w));
  // four columns at a time: their scales once for all rows, the quotients in the place of the elements
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 r = column_values(inv[0], lane8, j), d = column_values(inv[1], lane8, j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t &w = j == 0 ? raw[i].x : j == 1 ? raw[i].y : j == 2 ? raw[i].z : raw[i].w;
      const float2 a = unpack_fp8x2<XE5M2>(static_cast<uint16_t>(w)), b = unpack_fp8x2<XE5M2>(static_cast<uint16_t>(w >> 16));
      const float2 qa = quotients(mul2(a, both(-sx[i])), make_float2(d.x, d.y), make_float2(r.x, r.y));
      const float2 qb = quotients(mul2(b, both(-sx[i])), make_float2(d.z, d.w), make_float2(r.z, r.w));
      w = to_fp8x2<E5M2>(qa.x, qa.y) | to_fp8x2<E5M2>(qb.x, qb.y) << 16;
    }
  }
  unsigned char *q = p.q + r0 * p.ldq + c;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (32 * i < rows) store16_fp8(q + 32 * i * p.ldq, raw[i], n, level(vec, 1));
}

}  // namespace

cudaError_t launch_requantize(const RequantizeParams &p, cudaStream_t s) {
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = tiles_c * ((p.rows + 127) / 128);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const auto kernel = p.x_e5m2 ? p.e5m2 ? requantize_kernel<true, true> : requantize_kernel<true, false>
                      : p.e5m2 ? requantize_kernel<false, true>
                               : requantize_kernel<false, false>;
  return launch_maybe_pdl(kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, true, p,
                          static_cast<unsigned>(tiles_c), level_of(p.x, p.ldx, 1, 0) | level_of(p.q, p.ldq, 1, 1));
}

}  // namespace sg
