// fp8.cuh -- element types of the 8-bit linear layer's kernels: loads and
// stores of eight consecutive elements of F32, BF16, F16 and the 8-bit types,
// and the maximum that keeps NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"

namespace sg {

constexpr float kMaxE4m3 = 448.0f, kMaxE5m2 = 57344.0f;
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126: 1 / s is finite

// The larger of |a| and |b|; NaN if either is NaN (fmaxf would drop it).
__device__ __forceinline__ float max_abs(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

// Scale of a block whose largest |x| is a; s >= a / F, and a NaN or infinite a
// is the scale itself (fmaxf would drop the NaN).
__device__ __forceinline__ float block_scale(float a, bool e5m2) {
  const float s = __fdiv_rn(a, e5m2 ? kMaxE5m2 : kMaxE4m3);
  return s < kLeastScale ? kLeastScale : s;
}

// Two floats -> two 8-bit elements (x0 in the low byte), nearest even,
// saturating; NaN stays NaN.
template <bool E5M2>
__device__ __forceinline__ uint32_t to_fp8x2(float x0, float x1) {
  uint16_t r;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
// x / s from ninv = -1 / s: the product and one correction by its remainder, which an FMA gives exactly.
// The product alone is up to one and a half units in the last place off.  Where x has few bits its quotient by
// max / F often is a midpoint between two 8-bit values, which the product then leaves for the wrong side: of 42 million
// BF16 values in E4M3 21072 differed from the definition in 64 bits, 661 with the correction and with an FP32 division
// alike, which two agreed in every value (F16 2454 and 131; F32 24 and 21).
// Of -x and -1 / s, since a remainder of zero is then taken off a quotient of -0, which keeps its sign (with every
// sign the other way round it is added; negating the remainder instead cost 22.8 us for 21.3 at 4095 x 4104 both ways).
// s comes from divisor(): of an infinite scale it is 0, so that a finite x over it stays 0 (0 * inf would be NaN).
__device__ __forceinline__ float divisor(float scale) { return scale < INFINITY ? scale : 0.0f; }
__device__ __forceinline__ float quotient(float x, float s, float ninv) {
  const float nx = -x, q = nx * ninv;
  return fmaf(fmaf(q, s, nx), ninv, q);
}
__device__ __forceinline__ uint2 to_fp8x8(const float (&v)[8], float mul, bool e5m2) {
  uint2 u;
  if (e5m2) {
    u.x = to_fp8x2<true>(v[0] * mul, v[1] * mul) | to_fp8x2<true>(v[2] * mul, v[3] * mul) << 16;
    u.y = to_fp8x2<true>(v[4] * mul, v[5] * mul) | to_fp8x2<true>(v[6] * mul, v[7] * mul) << 16;
  } else {
    u.x = to_fp8x2<false>(v[0] * mul, v[1] * mul) | to_fp8x2<false>(v[2] * mul, v[3] * mul) << 16;
    u.y = to_fp8x2<false>(v[4] * mul, v[5] * mul) | to_fp8x2<false>(v[6] * mul, v[7] * mul) << 16;
  }
  return u;
}
// Eight elements of one block.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float s, float ninv, bool e5m2) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, ninv);
  return to_fp8x8(q, 1.0f, e5m2);
}

// ------------------------------------------------------------ F32, BF16, F16
// Raw<T>: eight consecutive elements as loaded.
template <class T> struct Raw;
template <> struct Raw<float> { uint4 u[2]; };
template <> struct Raw<__nv_bfloat16> { uint4 u[1]; };
template <> struct Raw<__half> { uint4 u[1]; };

__device__ __forceinline__ void unpack(const Raw<float> &r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.u[i].x);
    v[4 * i + 1] = __uint_as_float(r.u[i].y);
    v[4 * i + 2] = __uint_as_float(r.u[i].z);
    v[4 * i + 3] = __uint_as_float(r.u[i].w);
  }
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float (&v)[8]) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<__half> &r, float (&v)[8]) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void pack(Raw<float> &r, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.u[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                        __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <class T>
__device__ __forceinline__ void pack(Raw<T> &r, const float (&v)[8]) {
  r.u[0] = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                      pack2(v[6], v[7], T()));
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float *p, float x) { *p = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(__half *p, float x) { *p = __float2half_rn(x); }

// Elements p[0 .. n-1] (n <= 8; zeros beyond, nothing read there); `vec`: the
// rows are 16-byte aligned, so eight whole elements are one or two vectors.
// Ordinary loads: the kernel may have been resident while its predecessor
// wrote these elements, which the read-only path must not assume away.
template <class T>
__device__ __forceinline__ Raw<T> load8(const T *p, int n, bool vec) {
  Raw<T> r;
  if (n >= 8 && vec) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i)
      r.u[i] = reinterpret_cast<const uint4 *>(p)[i];
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_float(p[i]) : 0.0f;
    pack(r, v);   // exact: the values came from T
  }
  return r;
}
template <class T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8], int n, bool vec) {
  if (n >= 8 && vec) {
    Raw<T> r;
    pack(r, v);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) reinterpret_cast<uint4 *>(p)[i] = r.u[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) from_float(p + i, v[i]);
  }
}
// Eight 8-bit elements; vec: p is 8-byte aligned.
__device__ __forceinline__ void store8_fp8(unsigned char *p, uint2 u, int n, bool vec) {
  if (n >= 8 && vec) {
    *reinterpret_cast<uint2 *>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<unsigned char>((i < 4 ? u.x : u.y) >> (8 * (i & 3)));
  }
}

inline __host__ __device__ bool aligned_rows(const void *p, int64_t ld, int elem, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * elem) % bytes == 0;
}

}  // namespace sg
