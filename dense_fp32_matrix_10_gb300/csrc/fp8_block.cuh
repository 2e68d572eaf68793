// fp8_block.cuh -- what the kernels around a gated block's products share.
//
// They move 2 to 10 bytes an element and have some 15 to 45 instructions for
// it before they are bound by their issue slots instead of by memory.  So a
// lane holds 16 consecutive elements (eight lanes a block of 128), products
// and sums go two at a time, maxima three at a time, and the scales of several
// blocks are found together.
#pragma once

#include "fp8.cuh"
#include "fp8_block.h"

namespace sg {

// ------------------------------------------------------------ alignment
// How a call's rows are aligned, two bits an array: float types 2 = 32 bytes,
// 1 = 16 bytes; 8-bit types 2 = 16 bytes, 1 = 8 bytes.
__device__ __forceinline__ int level(uint32_t vec, int i) { return vec >> (2 * i) & 3; }
inline uint32_t level_of(const void *p, int64_t ld, int elem, int i) {
  const int wide = elem == 1 ? 16 : 32;
  return (aligned_rows(p, ld, elem, wide) ? 2u : aligned_rows(p, ld, elem, wide / 2) ? 1u : 0u) << (2 * i);
}

// ------------------------------------------------------------ sixteen elements of F32, BF16 or F16
template <class T>
struct Raw16 {
  Raw<T> half[2];
};
__device__ __forceinline__ void load_32(uint4 *u, const void *p) {   // 32 bytes on their alignment
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0].x), "=r"(u[0].y), "=r"(u[0].z), "=r"(u[0].w), "=r"(u[1].x), "=r"(u[1].y), "=r"(u[1].z), "=r"(u[1].w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_32(void *p, const uint4 *u) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0].x), "r"(u[0].y), "r"(u[0].z),
               "r"(u[0].w), "r"(u[1].x), "r"(u[1].y), "r"(u[1].z), "r"(u[1].w)
               : "memory");
}
// Whether the 16-byte units around the elements c .. c + 15 of a row lie in it whatever its alignment (c: a multiple of 16).
template <class C>
__device__ __forceinline__ bool inside(C c, C cols) { return c >= 16 && c + 24 <= cols; }
// Sixteen elements off 16 bytes, from the aligned units around them: their 32-bit words moved down by up to three, then
// their bytes.  (4000 x 4001 bf16, so and with the inputs and outputs element by element: norms with checkpoints 48 and 139
// us, their gradient 70 and 231, the unit 32 and 43, its gradient 54 and 58.)
template <class T>
__device__ __forceinline__ Raw16<T> load16_across(const T *p) {
  constexpr int W = 4 * static_cast<int>(sizeof(T));   // words
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint4 *from = reinterpret_cast<const uint4 *>(at & ~static_cast<uintptr_t>(15));
  uint32_t w[W + 4];
#pragma unroll
  for (int i = 0; i < W / 4 + 1; ++i) {
    const uint4 u = from[i];
    w[4 * i] = u.x;
    w[4 * i + 1] = u.y;
    w[4 * i + 2] = u.z;
    w[4 * i + 3] = u.w;
  }
  const bool two = at & 8, one = at & 4;
#pragma unroll
  for (int i = 0; i < W + 2; ++i) w[i] = two ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < W + 1; ++i) w[i] = one ? w[i + 1] : w[i];
  if (sizeof(T) == 2) {
    const int bits = static_cast<int>(at & 2) * 8;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  }
  Raw16<T> r;
#pragma unroll
  for (int i = 0; i < W / 4; ++i)
    r.half[i / (sizeof(T) / 2)].u[i % (sizeof(T) / 2)] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  return r;
}
// p[0 .. n-1] (zeros beyond); nothing outside is read, but where `in` says that it is of the same row (see inside()).
template <class T>
__device__ __forceinline__ Raw16<T> load16(const T *p, int n, int level, bool in = false) {
  Raw16<T> r;
  if (n >= 16 && level == 2) {
    uint4 u[sizeof(T)];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); i += 2) load_32(u + i, reinterpret_cast<const uint4 *>(p) + i);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) r.half[i / (sizeof(T) / 2)].u[i % (sizeof(T) / 2)] = u[i];
  } else if (level == 0 && in) {
    r = load16_across(p);
  } else {
    // (lanes behind a row's end skip it: norms 4000 x 4000 bf16 with checkpoints 38 us, else 44)
    r.half[0] = n > 0 ? load8(p, n, level) : Raw<T>();
    r.half[1] = n > 8 ? load8(p + 8, n - 8, level) : Raw<T>();
  }
  return r;
}
__device__ __forceinline__ float2 unpack_pair(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack_pair(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ void unpack(const Raw16<float> &r, float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 u = r.half[i / 2].u[i % 2];
    v[2 * i] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    v[2 * i + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
}
template <class T>
__device__ __forceinline__ void unpack(const Raw16<T> &r, float2 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = r.half[i].u[0];
    v[4 * i] = unpack_pair(u.x, T());
    v[4 * i + 1] = unpack_pair(u.y, T());
    v[4 * i + 2] = unpack_pair(u.z, T());
    v[4 * i + 3] = unpack_pair(u.w, T());
  }
}
// All signs the other way round.
template <class T>
__device__ __forceinline__ Raw16<T> negated(const Raw16<T> &r) {
  constexpr uint32_t sign = sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
  Raw16<T> n;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T) / 2); ++j) {
      const uint4 u = r.half[i].u[j];
      n.half[i].u[j] = make_uint4(u.x ^ sign, u.y ^ sign, u.z ^ sign, u.w ^ sign);
    }
  return n;
}
template <class T>
__device__ __forceinline__ void store16(T *p, const float2 (&v)[8], int n, int level) {
  float f[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i / 4][2 * i % 8] = v[i].x;
    f[i / 4][2 * i % 8 + 1] = v[i].y;
  }
  if (n >= 16 && level == 2) {
    Raw<T> r[2];
    pack(r[0], f[0]);
    pack(r[1], f[1]);
    uint4 u[sizeof(T)];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) u[i] = r[i / (sizeof(T) / 2)].u[i % (sizeof(T) / 2)];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); i += 2) store_32(reinterpret_cast<uint4 *>(p) + i, u + i);
  } else {
    if (n > 0) store8(p, f[0], n, level);
    if (n > 8) store8(p + 8, f[1], n - 8, level);
  }
}
// Sixteen weights (or a gate's row) of F32 or T.
template <class T>
__device__ __forceinline__ void load16_w(const void *w, bool f32, int64_t c, int n, int level, float2 (&v)[8]) {
  if (f32)
    unpack(load16(static_cast<const float *>(w) + c, n, level), v);
  else
    unpack(load16(static_cast<const T *>(w) + c, n, level), v);
}

// ------------------------------------------------------------ sixteen 8-bit elements
__device__ __forceinline__ uint2 load8_fp8(const unsigned char *p, int n, bool vec) {
  if (n >= 8 && vec) return *reinterpret_cast<const uint2 *>(p);
  uint2 u = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) (i < 4 ? u.x : u.y) |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return u;
}
__device__ __forceinline__ uint4 load16_fp8(const unsigned char *p, int n, int level) {
  if (n >= 16 && level == 2) return *reinterpret_cast<const uint4 *>(p);
  const uint2 a = n > 0 ? load8_fp8(p, n, level) : make_uint2(0, 0), b = n > 8 ? load8_fp8(p + 8, n - 8, level) : make_uint2(0, 0);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store16_fp8(unsigned char *p, uint4 u, int n, int level) {
  if (n >= 16 && level == 2) {
    *reinterpret_cast<uint4 *>(p) = u;
  } else {
    if (n > 0) store8_fp8(p, make_uint2(u.x, u.y), n, level);
    if (n > 8) store8_fp8(p + 8, make_uint2(u.z, u.w), n - 8, level);
  }
}
// The first n of sixteen, zeros behind.
__device__ __forceinline__ uint4 first16_fp8(uint4 u, int n) {
  const auto word = [&](uint32_t w, int m) { return m >= 4 ? w : m > 0 ? w & ((1u << 8 * m) - 1) : 0u; };
  return n >= 16 ? u : make_uint4(word(u.x, n), word(u.y, n - 4), word(u.z, n - 8), word(u.w, n - 12));
}
// (exact)
template <bool E5M2>
__device__ __forceinline__ float2 unpack_fp8x2(uint16_t two) {
  uint32_t h;
  if (E5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(two));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
template <bool E5M2>
__device__ __forceinline__ void unpack_fp8(uint4 u, float2 (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = unpack_fp8x2<E5M2>(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
}
template <bool E5M2>
__device__ __forceinline__ uint4 to_fp8x16(const float2 (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = to_fp8x2<E5M2>(v[2 * i].x, v[2 * i].y) | to_fp8x2<E5M2>(v[2 * i + 1].x, v[2 * i + 1].y) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------ asynchronous copies
// Sixteen bytes (or four) of this thread's own, to a place in shared memory that it alone uses.
__device__ __forceinline__ void copy_16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// The first `bytes` of them (0 .. 16), zeros behind.
__device__ __forceinline__ void copy_16(void *dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most n of this thread's groups are in flight.
__device__ __forceinline__ void copies_wait(int n) {
  if (n <= 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
}
// A thread's 16-byte units lie a warp's width apart: no bank conflicts, and constant offsets from its first.
constexpr int kUnitStep = 32;
__device__ __forceinline__ int first_unit(int units) {   // of this thread, where each has `units` of them
  return (threadIdx.x >> 5) * units * kUnitStep + (threadIdx.x & 31);
}
// The first n (1 .. 16) of sixteen elements of T on 16 bytes, zeros behind, in sizeof(T) units.
template <class T>
__device__ __forceinline__ void copy16_first(uint4 *to, const T *x, int n) {
  constexpr int U = sizeof(T);
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int bytes = max(0, min(n * U - 16 * k, 16));
    copy_16(to + k * kUnitStep, reinterpret_cast<const uint4 *>(x) + (bytes ? k : 0), bytes);   // (no address behind the row)
  }
}
// n of any count and alignment: a row's end is copied like the rest of it where it is aligned, without a wait (4000 x 4008
// bf16, the norms' gradient: 49 us, element by element 65).
template <class T>
__device__ __forceinline__ void copy16(uint4 *to, const T *x, int n, int level, bool in = false) {
  constexpr int U = sizeof(T);
  if (n >= 16 && level) {
#pragma unroll
    for (int k = 0; k < U; ++k) copy_16(to + k * kUnitStep, reinterpret_cast<const uint4 *>(x) + k);
  } else if (n > 0 && level) {
    copy16_first(to, x, n);
  } else {
    const Raw16<T> r = load16(x, n, level, in);
#pragma unroll
    for (int k = 0; k < U; ++k) to[k * kUnitStep] = r.half[k / (U / 2)].u[k % (U / 2)];
  }
}
template <class T>
__device__ __forceinline__ Raw16<T> take16(const uint4 *at) {
  constexpr int U = sizeof(T);
  Raw16<T> r;
#pragma unroll
  for (int k = 0; k < U; ++k) r.half[k / (U / 2)].u[k % (U / 2)] = at[k * kUnitStep];
  return r;
}
// Sixteen elements of a checkpoint, one unit, and their scale.
__device__ __forceinline__ void copy16_kept(uint4 *to, float *scale, const unsigned char *x, const float *s, int n, int level) {
  if (n >= 16 && level == 2)
    copy_16(to, x);
  else if (n > 0 && level == 2)
    copy_16(to, x, n);
  else
    *to = load16_fp8(x, n, level);
  if (n > 0)
    copy_4(scale, s);
  else
    *scale = 0.0f;
}

// ------------------------------------------------------------ packed FP32
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest magnitude of sixteen.
__device__ __forceinline__ float max_abs16(const float2 (&v)[8]) {
  float m = max_abs(v[0].x, v[0].y), k = max_abs(v[1].x, v[1].y);
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    m = max_abs3(m, v[i].x, v[i].y);
    k = max_abs3(k, v[i + 1].x, v[i + 1].y);
  }
  return max_abs(m, k);
}
__device__ __forceinline__ float rcp_approx(float a) {   // one unit in the last place; subnormals are 0
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(a));
  return d;
}

// Zeros for the elements from n on, whatever a row that holds a NaN or an infinity has made of those behind its end.
__device__ __forceinline__ void clear_from(float2 (&v)[8], int n) {
  if (n >= 16) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i >= n) v[i].x = 0.0f;
    if (2 * i + 1 >= n) v[i].y = 0.0f;
  }
}

// ------------------------------------------------------------ scales and quotients
// block_scale() in six instructions: a / F as a (1 / F), corrected by its remainder (which an FMA gives exactly down to
// the scales that are replaced by the least one).  Equal to the division: tested for every significand.
__device__ __forceinline__ float scale_of(float a, bool e5m2) {
  const float F = e5m2 ? kMaxE5m2 : kMaxE4m3, inv = e5m2 ? 1.0f / kMaxE5m2 : 1.0f / kMaxE4m3;
  const float q = a * inv;
  float s = fmaf(fmaf(-q, F, a), inv, q);
  s = a < INFINITY ? s : a;
  return s < kLeastScale ? kLeastScale : s;
}
// -1 / scale for quotients: their correction makes up for what it is off by.
__device__ __forceinline__ float ninv_of(float scale) { return -rcp_approx(scale); }

// The maxima of four sets of magnitudes, each over the eight lanes of a block: a lane passes on the half of its maxima
// that the other lane of a pair will own, then half of the rest; a third exchange joins the two lanes that own the same
// one.  4 exchanges instead of 12, and a scale's arithmetic once instead of four times.
__device__ __forceinline__ int owned_by(int lane8) { return (lane8 >> 2 & 1) * 2 + (lane8 >> 1 & 1); }
__device__ __forceinline__ constexpr int owner_of(int i) { return (i & 2) * 2 + (i & 1) * 2; }   // and the next lane
__device__ __forceinline__ float owned_max(const float (&v)[4], int lane8) {
  const bool h4 = lane8 & 4, h2 = lane8 & 2;
  float a[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) a[i] = max_abs(h4 ? v[2 + i] : v[i], __shfl_xor_sync(~0u, h4 ? v[i] : v[2 + i], 4));
  const float b = max_abs(h2 ? a[1] : a[0], __shfl_xor_sync(~0u, h2 ? a[0] : a[1], 2));
  return max_abs(b, __shfl_xor_sync(~0u, b, 1));
}
__device__ __forceinline__ float max_of_8(float a) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) a = max_abs(a, __shfl_xor_sync(~0u, a, d));
  return a;
}

// Quotients of what a caller knows (given values, and h), which often have few bits and then lie between two 8-bit values:
// x / s from -x, div = divisor(s) and ninv (see quotient()).
__device__ __forceinline__ float2 quotients(float2 nx, float2 div, float2 ninv) {
  const float2 q = mul2(nx, ninv);
  return fma2(fma2(q, div, nx), ninv, q);
}
template <bool E5M2>
__device__ __forceinline__ uint4 quantise_exactly(const float2 (&nx)[8], float div, float ninv) {
  float2 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotients(nx[i], both(div), both(ninv));
  return to_fp8x16<E5M2>(q);
}
// Quotients of values that are quantised as they are computed, which are themselves off by more than the product with the
// rounded 1 / s (0 for an infinite scale): a correction costs two more operations for each and brings them no nearer (as
// many 8-bit values differ from those in 64 bits; the unit's gradient 4095 x 8192 95 instead of 85 us, the unit 88.5 and 86).
__device__ __forceinline__ float inv_of(float scale) {
  const float r = rcp_approx(scale);
  const float e = fmaf(-scale, r, 1.0f);
  return scale < INFINITY ? fmaf(e, r, r) : r;
}
template <bool E5M2>
__device__ __forceinline__ uint4 quantise(const float2 (&x)[8], float inv) {
  float2 q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = mul2(x[i], both(inv));
  return to_fp8x16<E5M2>(q);
}
// Values for a tile's 128 columns in shared memory, so that eight lanes read those of four of their 16 columns without
// a bank conflict (in the columns' order, 64 bytes apart, four lanes would meet in a bank).
__device__ __forceinline__ int column_place(int col) { return ((col >> 2 & 3) * 8 + (col >> 4)) * 4 + (col & 3); }
__device__ __forceinline__ float4 column_values(const float *v, int lane8, int j) {
  return *reinterpret_cast<const float4 *>(v + (j * 8 + lane8) * 4);
}

}  // namespace sg
