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

// Maxima over 16 lanes of eight values each: a lane passes on the half of its values that the other
// lane of a pair will own, so three exchanges leave one value a lane and a fourth joins the two lanes
// that own the same one.  Lane l (of 16) ends with the maximum of value owned(l).
__device__ __forceinline__ int owned(int lane16) { return (lane16 >> 3 & 1) * 4 + (lane16 >> 2 & 1) * 2 + (lane16 >> 1 & 1); }
__device__ __forceinline__ float max_of_8x16(const float (&v)[8], int lane16) {
  float a[4], b[2];
  const bool h8 = lane16 & 8, h4 = lane16 & 4, h2 = lane16 & 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = max_abs(h8 ? v[4 + i] : v[i], __shfl_xor_sync(~0u, h8 ? v[i] : v[4 + i], 8));
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = max_abs(h4 ? a[2 + i] : a[i], __shfl_xor_sync(~0u, h4 ? a[i] : a[2 + i], 4));
  float c = max_abs(h2 ? b[1] : b[0], __shfl_xor_sync(~0u, h2 ? b[0] : b[1], 2));
  return max_abs(c, __shfl_xor_sync(~0u, c, 1));
}

template <class T, int MODE>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2)
    quantize_kernel(const QuantizeParams p, const int64_t tiles_c, const bool vec_x, const bool vec_r,
                    const bool vec_c) {
  __shared__ float part[8][128];   // column maxima of each warp, then of the tile
  griddep_wait();
  griddep_launch_dependents();
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
  const int64_t c0 = tc * 128 + lane16 * 8;
  const int64_t left = p.cols - c0;
  const int n = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
  const int64_t r0 = tr * 128 + row16;   // this thread's rows: r0 + 16 i
  const int rows = static_cast<int>(min(int64_t(128), p.rows - r0));
  Raw<T> raw[8];
  {
    const T *x = static_cast<const T *>(p.x) + r0 * p.ldx + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = load8(x + 16 * i * p.ldx, 16 * i < rows ? n : 0, vec_x);
  }
  float cmax[8], rmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[j] = rmax[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack(raw[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (MODE & kCol) cmax[j] = max_abs(cmax[j], v[j]);
      if (MODE & (kRow | kTile)) rmax[i] = max_abs(rmax[i], v[j]);
    }
  }
  if (MODE & kRow) {
    // each lane divides for the row that it owns
    const int mine = owned(lane16);
    const float s = block_scale(max_of_8x16(rmax, lane16), p.e5m2), ninv = __fdiv_rn(-1.0f, s), div = divisor(s);
    if ((lane16 & 1) == 0 && 16 * mine < rows) p.sr[(r0 + 16 * mine) * p.ldsr + tc] = s;
    unsigned char *q = p.qr + r0 * p.ldqr + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int from = (i & 4) * 2 + (i & 2) * 2 + (i & 1) * 2;
      const float si = __shfl_sync(~0u, div, from, 16), fi = __shfl_sync(~0u, ninv, from, 16);
      float v[8];
      unpack(raw[i], v);
      if (16 * i < rows) store8_fp8(q + 16 * i * p.ldqr, quantize8(v, si, fi, p.e5m2), n, vec_r);
    }
  }
  if (MODE & kTile) {
    float tmax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) tmax = max_abs(tmax, rmax[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) tmax = max_abs(tmax, __shfl_xor_sync(~0u, tmax, d));
    if ((threadIdx.x & 31) == 0) part[0][warp] = tmax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) tmax = max_abs(tmax, part[0][w]);
    const float s = block_scale(tmax, p.e5m2), ninv = __fdiv_rn(-1.0f, s);
    if (threadIdx.x == 0) p.sr[tr * p.ldsr + tc] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      unpack(raw[i], v);
      if (16 * i < rows)
        store8_fp8(p.qr + (r0 + 16 * i) * p.ldqr + c0, quantize8(v, divisor(s), ninv, p.e5m2), n, vec_r);
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
      part[0][threadIdx.x] = __fdiv_rn(-1.0f, s);
      part[1][threadIdx.x] = divisor(s);
    }
    __syncthreads();
    float ninv[8], scale[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ninv[j] = part[0][lane16 * 8 + j];
      scale[j] = part[1][lane16 * 8 + j];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = quotient(v[j], scale[j], ninv[j]);
      if (16 * i < rows)
        store8_fp8(p.qc + (r0 + 16 * i) * p.ldqc + c0, to_fp8x8(v, 1.0f, p.e5m2), n, vec_c);
    }
  }
}

// Both quantisations of 16-bit elements.  In registers (as above) the tile, its maxima and their use took 117
// registers and two CTAs an SM, too few bytes in flight (16384 x 8192 116 us, 4.6 TB/s); here the tile lies in
// shared memory, put there by asynchronous copies, and five CTAs fit (92 us; 108 with the corrected quotients that
// both forms have since).  Of F32, whose tile takes twice the room, the registers are as fast (4096 x 8192 38
// against 42 us).
template <class T>
__global__ void __launch_bounds__(256, 5)
    quantize_both_kernel(const QuantizeParams p, const int64_t tiles_c, const bool vec_x, const bool vec_r,
                         const bool vec_c) {
  constexpr int PITCH = 128 + 16 / sizeof(T);   // a 16-byte unit more: rows start in different banks
  extern __shared__ __align__(16) unsigned char tile_smem[];
  T *tile = reinterpret_cast<T *>(tile_smem);
  __shared__ __align__(16) float part[8][128];   // column maxima of 16 rows, then (part[0], part[1]) -1 / scale and scale
  griddep_wait();
  griddep_launch_dependents();
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int lane16 = threadIdx.x & 15, row16 = threadIdx.x >> 4;
  const int64_t c0 = tc * 128 + lane16 * 8, r0 = tr * 128 + row16;   // this thread's rows: r0 + 16 i
  const int64_t left = p.cols - c0;
  const int n = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
  const int rows = static_cast<int>(min(int64_t(128), p.rows - r0));
  T *mine = tile + row16 * PITCH + lane16 * 8;
  {
    const T *x = static_cast<const T *>(p.x) + r0 * p.ldx + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = 16 * i < rows ? n : 0;
      if (k == 8 && vec_x) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(mine + 16 * i * PITCH)),
                     "l"(x + 16 * i * p.ldx)
                     : "memory");
      } else {
        float v[8];
        unpack(load8(x + 16 * i * p.ldx, k, false), v);
        store8(mine + 16 * i * PITCH, v, 8, true);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncthreads();
  // maxima of 16 rows by 4 columns
  {
    const int c = (threadIdx.x & 31) * 4, r = (threadIdx.x >> 5) * 16;
    float m[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const T *x = tile + (r + i) * PITCH + c;
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max_abs(m[j], to_float(x[j]));
    }
    *reinterpret_cast<float4 *>(&part[threadIdx.x >> 5][c]) = make_float4(m[0], m[1], m[2], m[3]);
  }
  float rmax[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack(load8(mine + 16 * i * PITCH, 8, true), v);
    rmax[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) rmax[i] = max_abs(rmax[i], v[j]);
  }
  const int own = owned(lane16);
  const float s = block_scale(max_of_8x16(rmax, lane16), p.e5m2), row_ninv = __fdiv_rn(-1.0f, s), div = divisor(s);
  if ((lane16 & 1) == 0 && 16 * own < rows) p.sr[(r0 + 16 * own) * p.ldsr + tc] = s;
  __syncthreads();
  if (threadIdx.x < 128) {
    float a = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) a = max_abs(a, part[w][threadIdx.x]);
    const float t = block_scale(a, p.e5m2);
    const int64_t c = tc * 128 + threadIdx.x;
    if (c < p.cols) p.sc[tr * p.ldsc + c] = t;
    part[0][threadIdx.x] = __fdiv_rn(-1.0f, t);
    part[1][threadIdx.x] = divisor(t);
  }
  __syncthreads();
  float ninv[8], scale[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    ninv[j] = part[0][lane16 * 8 + j];
    scale[j] = part[1][lane16 * 8 + j];
  }
  unsigned char *qr = p.qr + r0 * p.ldqr + c0, *qc = p.qc + r0 * p.ldqc + c0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int from = (i & 4) * 2 + (i & 2) * 2 + (i & 1) * 2;
    const float si = __shfl_sync(~0u, div, from, 16), fi = __shfl_sync(~0u, row_ninv, from, 16);
    float v[8];
    unpack(load8(mine + 16 * i * PITCH, 8, true), v);
    if (16 * i < rows) {
      store8_fp8(qr + 16 * i * p.ldqr, quantize8(v, si, fi, p.e5m2), n, vec_r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = quotient(v[j], scale[j], ninv[j]);
      store8_fp8(qc + 16 * i * p.ldqc, to_fp8x8(v, 1.0f, p.e5m2), n, vec_c);
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
  if (p.qr && p.qc) {
    if constexpr (sizeof(T) == 4) {
      return go(quantize_kernel<T, kRow | kCol>);
    } else {
      constexpr int smem = 128 * (128 * static_cast<int>(sizeof(T)) + 16);
      return launch_maybe_pdl(quantize_both_kernel<T>, grid, block, smem, s, true, p, tiles_c, vx, vr, vc);
    }
  }
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
