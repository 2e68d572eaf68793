// sandwich_norm.cuh -- what the norms around a block and their gradient share.
//
//   tp = 1 / sqrt(mean a^2 + eps),  h = rho x + gate (a tp wp)
//   t  = 1 / sqrt(mean h^2 + eps),  y = h t w,  (q, s) = y in 1 x 128 blocks
//
//   H  = t (dy w - h t^2 mean(dy w h)) + dh,  dx = rho H
//   v  = H gate wp,  da = tp (v - a tp^2 mean(v a))
//   dw = sum dy h t,  dwp = sum H gate a tp,  dgate = wp sum H a tp
//
// A CTA takes consecutive rows, one at a time, 16 consecutive elements a
// thread; its weights stay in registers.  A thread copies its own elements of
// the next rows to places of its own in shared memory, so that memory is busy
// during a row's sums.  512 threads an SM with 128 registers each: one CTA for
// rows of 8192 elements, more of them for shorter ones.  Longer rows are walked
// in segments, several times.
#pragma once

#include <mutex>

#include "dispatch.h"
#include "fp8_block.cuh"

namespace sg {

constexpr int kRowThreads = 512, kRowElements = 16 * kRowThreads;
constexpr int kRowSmem = 208 * 1024;   // of an SM for the copied rows

// The sum over a CTA's threads, in a fixed order.  `red` is used by turns (`turn` flips with each call), so one barrier a
// call is enough.
__device__ __forceinline__ float row_total(float v, float (*red)[16], int &turn) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < blockDim.x >> 5 ? red[turn][lane] : 0.0f;   // at most 16 warps
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  turn ^= 1;
  return __shfl_sync(~0u, v, 0);
}
// Of three values: a lane passes on the two of four that the other lane of a pair will own, then one of two, and the
// eight lanes of an owner are joined (6 exchanges instead of 15); the warps' sums likewise.
__device__ __forceinline__ void row_totals(float &a, float &b, float &c, float (*red)[4][16], int &turn) {
  const int lane = threadIdx.x & 31, own = lane >> 3;
  const bool h16 = lane & 16, h8 = lane & 8;
  const float u = (h16 ? c : a) + __shfl_xor_sync(~0u, h16 ? a : c, 16);
  const float w = (h16 ? 0.0f : b) + __shfl_xor_sync(~0u, h16 ? b : 0.0f, 16);
  float v = (h8 ? w : u) + __shfl_xor_sync(~0u, h8 ? u : w, 8);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  if (blockDim.x > 32) {
    const unsigned warps = blockDim.x >> 5;
    if ((lane & 7) == 0) red[turn][own][threadIdx.x >> 5] = v;
    __syncthreads();
    v = ((lane & 7) < warps ? red[turn][own][lane & 7] : 0.0f) + ((lane & 7) + 8 < warps ? red[turn][own][(lane & 7) + 8] : 0.0f);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    turn ^= 1;
  }
  a = __shfl_sync(~0u, v, 0);
  b = __shfl_sync(~0u, v, 8);
  c = __shfl_sync(~0u, v, 16);
}

// CTAs, each with `rows` consecutive rows (the last one fewer).
struct Split {
  unsigned ctas, rows;
};
// Threads of a row's CTA, and how many of them an SM takes (512 threads).
struct RowsShape {
  int threads, per_sm;
  bool segments;
  Split split;
};
inline RowsShape rows_shape(int64_t rows, int64_t cols, int sm_count) {
  const int64_t chunks = (cols + 15) / 16;
  RowsShape g;
  g.segments = chunks > kRowThreads;
  g.threads = g.segments ? kRowThreads : static_cast<int>((chunks + 31) / 32 * 32);
  g.per_sm = kRowThreads / g.threads;
  const int64_t most = static_cast<int64_t>(sm_count) * g.per_sm;
  g.split.rows = rows > 0 ? static_cast<unsigned>((rows + most - 1) / most) : 1;
  g.split.ctas = static_cast<unsigned>((rows + g.split.rows - 1) / g.split.rows);
  return g;
}
// Rows in shared memory: as many as the SM's CTAs find room for, up to four.
inline int rows_ahead(const RowsShape &g, int row_bytes) {
  const int fit = kRowSmem / g.per_sm / row_bytes;
  return fit < 1 ? 1 : fit < 4 ? fit : 4;
}
// Once for each kernel (each has its own Tag) and device: all the shared memory that a launch may ask for.
template <class Tag, class F>
cudaError_t allow_smem(F *kernel) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [dev, kernel] {
    set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowSmem);
  });
  return set[dev];
}

}  // namespace sg
