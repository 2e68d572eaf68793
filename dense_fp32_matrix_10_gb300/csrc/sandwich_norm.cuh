// sandwich_norm.cuh -- what the norms around a block and their gradient share.
//
//   tp = 1 / sqrt(mean a^2 + eps),  h = rho x + gate (a tp wp)
//   t  = 1 / sqrt(mean h^2 + eps),  y = h t w,  (q, s) = y in 1 x 128 blocks
//
//   H  = t (dy w - h t^2 mean(dy w h)) + dh,  dx = rho H
//   v  = H gate wp,  da = tp (v - a tp^2 mean(v a))
//   dw = sum dy h t,  dwp = sum H gate a tp,  dgate = wp sum H a tp
//
// Both take a row into registers once, 16 consecutive elements a thread, and
// have an SM work on several rows: while some wait for a sum, stores or loads,
// another computes.  (With rows copied ahead through shared memory and one CTA of
// 512 threads an SM all its warps were in one phase, and the times of copies,
// arithmetic and stores added up: norms of 8192 x 8192 with checkpoints 43, 67
// and 32 us, 142 in all.)  Rows of more than 16384 elements are walked in
// segments, several times.
#pragma once

#include "dispatch.h"
#include "fp8_block.cuh"

namespace sg {

constexpr int kRowThreads = 1024, kRowElements = 16 * kRowThreads;   // of a row, or of a segment of a longer one
constexpr int kPairThreads = 256;                                    // of a row with twice 16 elements a thread

// Sums of K values (1 or 4) over a row's threads, in a fixed order.  A lane passes on the half of its values that the
// other lane of a pair will own, then half of the rest, until each owns one; the lanes that own the same one are joined
// (6 exchanges instead of 20).  The warps' sums likewise.  Used by turns, so that one barrier a call is enough.  Rows of
// one warp have blockDim.x == 32 and may share a CTA.
template <int K>
class RowSums {
  static_assert(K == 1 || K == 4, "");
  float (*red)[K][32];
  int turn = 0;

 public:
  __device__ __forceinline__ explicit RowSums(float (*shared)[K][32]) : red(shared) {
    if (blockDim.x == 32) return;
    for (int i = threadIdx.x; i < 2 * K * 32; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;   // absent warps' entries
    __syncthreads();
  }
  __device__ __forceinline__ void operator()(float (&v)[K]) {
    constexpr int G = 32 / K;   // lanes that own the same value
    const int lane = threadIdx.x & 31, own = lane / G;
#pragma unroll
    for (int k = K / 2, d = 16; k > 0; k >>= 1, d >>= 1) {
      const bool upper = lane & d;
#pragma unroll
      for (int i = 0; i < k; ++i) {
        const float mine = upper ? v[k + i] : v[i], give = upper ? v[i] : v[k + i];
        v[i] = mine + __shfl_xor_sync(~0u, give, d);
      }
    }
    float s = v[0];
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    if (blockDim.x > 32) {
      if (lane % G == 0) red[turn][own][threadIdx.x >> 5] = s;
      __syncthreads();
      const float *at = &red[turn][own][lane % G * (32 / G)];
      s = at[0];
#pragma unroll
      for (int i = 1; i < 32 / G; ++i) s += at[i];
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      turn ^= 1;
    }
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = __shfl_sync(~0u, s, i * G);
  }
};

// Threads of a row (a multiple of 32, at most 1024).
inline int row_threads(int64_t cols) {
  const int64_t chunks = (cols + 15) / 16;
  return static_cast<int>(chunks > kRowThreads ? kRowThreads : (chunks + 31) / 32 * 32);
}

}  // namespace sg
