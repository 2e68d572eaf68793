// fp8_block.cuh -- what the kernels around a gated block's products share:
// reading checkpoints, and quantising blocks whose values lie in registers.
#pragma once

#include "fp8.cuh"
#include "fp8_block.h"

namespace sg {

// Eight 8-bit elements as floats (exact).
__device__ __forceinline__ void unpack_fp8(uint2 u, bool e5m2, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t two = static_cast<uint16_t>((i < 2 ? u.x : u.y) >> (16 * (i & 1)));
    uint32_t h;
    if (e5m2)
      asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(two));
    else
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// p[0 .. n-1] (n <= 8; zeros beyond, nothing read there); vec: p is 8-byte aligned.
__device__ __forceinline__ uint2 load8_fp8(const unsigned char *p, int n, bool vec) {
  if (n >= 8 && vec) return *reinterpret_cast<const uint2 *>(p);
  uint2 u = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) (i < 4 ? u.x : u.y) |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return u;
}

// The maximum over the 16 lanes that hold a block.
__device__ __forceinline__ float max_of_16(float a) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) a = max_abs(a, __shfl_xor_sync(~0u, a, d));
  return a;
}
// Quantises eight of a block's values (the other 15 lanes hold the rest; the first n are the matrix'), and its scale.
__device__ __forceinline__ void store_block(const float (&v)[8], int n, unsigned char *q, float *s, bool e5m2, bool vec) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) a = max_abs(a, v[i]);
  const float scale = block_scale(max_of_16(a), e5m2);
  store8_fp8(q, quantize8(v, divisor(scale), __fdiv_rn(-1.0f, scale), e5m2), n, vec);
  if ((threadIdx.x & 15) == 0 && n > 0) *s = scale;
}

}  // namespace sg
