// row_norm.cuh -- what the kernels that normalise rows share: the sum over a
// row's threads, its weights, and how a row is laid over threads.
//
// A row is held by `G` threads, eight consecutive elements at a time (chunk
// j * G + thread), so the 16 threads of half a warp hold one block of 128.
#pragma once

#include "fp8.cuh"

namespace sg {

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Sum over the threads of a row: over the warp (blockDim.x == 32: one row per
// warp), or over the CTA (blockDim.y == 1), in a fixed order.  `red` is used
// by turns (`turn` flips with each call), so one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int &turn) {
  v = warp_sum(v);
  if (blockDim.x == 32) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = warp_sum(lane < warps ? red[turn][lane] : 0.0f);
  turn ^= 1;
  return v;
}

// Eight weights as floats.
template <class T>
__device__ __forceinline__ void load_w(const void *w, bool f32, int64_t c, int n, bool vec, float (&v)[8]) {
  if (f32)
    unpack(load8(static_cast<const float *>(w) + c, n, vec), v);
  else
    unpack(load8(static_cast<const T *>(w) + c, n, vec), v);
}

// Threads of a row and chunks of eight a thread holds.
struct RowShape {
  int threads, nv, rows;   // rows per CTA (threads == 32 only)
  bool loop;
};
inline RowShape row_shape(int64_t rows, int64_t cols, int sm_count) {
  const int64_t chunks = (cols + 7) / 8;
  auto up32 = [](int64_t v) { return static_cast<int>((v + 31) / 32 * 32); };
  if (chunks <= 32) return {32, 1, 8, false};
  if (chunks <= 128 && rows >= 4 * sm_count) return {32, chunks <= 64 ? 2 : 4, 8, false};
  // few rows: as many threads as there are chunks, for the shortest chain
  if (chunks <= kMaxThreads && rows <= 2 * sm_count) return {up32(chunks), 1, 1, false};
  if (chunks <= 2 * 512) return {up32((chunks + 1) / 2), 2, 1, false};
  if (chunks <= 4 * 512) return {up32((chunks + 3) / 4), 4, 1, false};
  return {512, 4, 1, true};
}

}  // namespace sg
