// rms_norm.cu -- RMS norm of x + r with a quantised output, and its gradient.
//
//   h = x + r,  t = 1 / sqrt(mean h^2 + eps),  y = h t w,  (q, s) = y in 1 x 128 blocks
//   g = dy w,   dx = t (g - h t^2 mean(g h)) + dh,   dw = sum over rows of dy h t
//
// A row is held by `G` threads, eight consecutive elements at a time (chunk
// j * G + thread), so the 16 threads of half a warp hold one block of 128 and
// its maximum is four shuffles.  A row of up to 8 * G * NV elements stays in
// registers between the statistics and the output: x and r are read once.
// Longer rows are walked in segments and read a second time.
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace sg {
namespace {

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

// vec: bit 0 x, 1 r, 2 w, 3 h, 4 y (16-byte rows), 5 q (8-byte rows)
template <class T, int NV, bool LONG>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) rms_norm_kernel(const NormParams p, const int vec) {
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;   // whole warps: a CTA of several warps per row has blockDim.y == 1
  const T *x = static_cast<const T *>(p.x) + row * p.ldx;
  const T *r = p.r ? static_cast<const T *>(p.r) + row * p.ldr : nullptr;
  const int64_t seg = static_cast<int64_t>(8) * NV * blockDim.x;
  float h[NV][8];
  int turn = 0;
  auto load = [&](int64_t base) {
    Raw<T> a[NV], b[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = base + (static_cast<int64_t>(j) * blockDim.x + threadIdx.x) * 8;
      const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c)));
      a[j] = load8(x + c, n, vec & 1);
      if (r) b[j] = load8(r + c, n, vec & 2);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack(a[j], h[j]);
      if (r) {
        float v[8];
        unpack(b[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] += v[i];
      }
    }
  };
  float sum = 0.0f;
  for (int64_t base = 0; base < (LONG ? p.cols : 1); base += seg) {
    load(base);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += h[j][i] * h[j][i];
  }
  sum = row_sum(sum, red, turn);
  const float t = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  if (p.t && threadIdx.x == 0) p.t[row] = t;
  for (int64_t base = 0; base < (LONG ? p.cols : 1); base += seg) {
    if (LONG) load(base);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = base + (static_cast<int64_t>(j) * blockDim.x + threadIdx.x) * 8;
      const int n = static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c)));
      if (p.h) store8(static_cast<T *>(p.h) + row * p.ldh + c, h[j], n, vec & 8);
      float w[8], y[8], a = 0.0f;
      load_w<T>(p.w, p.w_f32, c, n, vec & 4, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = h[j][i] * t * w[i];
        if (i < n) a = max_abs(a, y[i]);   // a NaN or infinite t must not reach past the row's end
      }
      if (p.y) store8(static_cast<T *>(p.y) + row * p.ldy + c, y, n, vec & 16);
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) a = max_abs(a, __shfl_xor_sync(~0u, a, d));
      const float s = block_scale(a, p.e5m2);
      store8_fp8(p.q + row * p.ldq + c, to_fp8x8(y, __fdiv_rn(1.0f, s), p.e5m2), n, vec & 32);
      if ((threadIdx.x & 15) == 0 && n > 0) p.s[row * p.lds + c / 128] = s;
    }
  }
}

// CTA b takes rows b, b + grid, ... and adds dy h t of its rows per column in
// registers (LONG: in its row of the workspace).
template <class T, int NV, bool LONG>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512)
    rms_norm_backward_kernel(const NormGradParams p, const int vec) {
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t seg = static_cast<int64_t>(8) * NV * blockDim.x, pitch = (p.cols + 7) / 8 * 8;
  float dw[NV][8], dy[NV][8], h[NV][8], w[NV][8];
  int turn = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  auto at = [&](int64_t base, int j, int &n) {
    const int64_t c = base + (static_cast<int64_t>(j) * blockDim.x + threadIdx.x) * 8;
    n = static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c)));
    return c;
  };
  auto load_weights = [&](int64_t base) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      int n;
      const int64_t c = at(base, j, n);
      load_w<T>(p.w, p.w_f32, c, n, vec & 4, w[j]);
    }
  };
  auto load = [&](int64_t row, int64_t base) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      int n;
      const int64_t c = at(base, j, n);
      unpack(load8(static_cast<const T *>(p.dy) + row * p.lddy + c, n, vec & 1), dy[j]);
      unpack(load8(static_cast<const T *>(p.h) + row * p.ldh + c, n, vec & 2), h[j]);
    }
  };
  if (!LONG) load_weights(0);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float t = p.t[row];
    float sum = 0.0f;
    for (int64_t base = 0; base < (LONG ? p.cols : 1); base += seg) {
      load(row, base);
      if (LONG) load_weights(base);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += dy[j][i] * w[j][i] * h[j][i];
    }
    sum = row_sum(sum, red, turn);
    const float k = t * t * (sum / static_cast<float>(p.cols));
    for (int64_t base = 0; base < (LONG ? p.cols : 1); base += seg) {
      if (LONG) {
        load(row, base);
        load_weights(base);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        int n;
        const int64_t c = at(base, j, n);
        float v[8];
        if (p.dh) unpack(load8(static_cast<const T *>(p.dh) + row * p.lddh + c, n, vec & 8), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = t * (dy[j][i] * w[j][i] - h[j][i] * k);
          v[i] = p.dh ? v[i] + d : d;
        }
        store8(static_cast<T *>(p.dx) + row * p.lddx + c, v, n, vec & 16);
        if (LONG && p.partial && n > 0) {   // this CTA's own row: no other thread touches these
          float *mine = p.partial + blockIdx.x * pitch + c;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mine[i] = (row == blockIdx.x ? 0.0f : mine[i]) + dy[j][i] * h[j][i] * t;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dw[j][i] += dy[j][i] * h[j][i] * t;
        }
      }
    }
  }
  if (LONG || !p.partial) return;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    int n;
    const int64_t c = at(0, j, n);
    if (n > 0) store8(p.partial + blockIdx.x * pitch + c, dw[j], 8, true);
  }
}

// dw[c] = sum over the CTAs' partial rows, in their order.
template <class T>
__global__ void __launch_bounds__(256) norm_dw_kernel(const float *partial, int parts, int64_t cols, T *dw) {
  __shared__ float red[8][32];
  griddep_wait();
  const int64_t pitch = (cols + 7) / 8 * 8;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < cols)
    for (int i = threadIdx.y; i < parts; i += 8) v += partial[i * pitch + c];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][threadIdx.x];
    from_float(dw + c, v);
  }
}

// Threads of a row and chunks of eight a thread holds.
struct RowShape {
  int threads, nv, rows;   // rows per CTA (threads == 32 only)
  bool loop;
};
RowShape row_shape(int64_t rows, int64_t cols, int sm_count) {
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

template <class T>
cudaError_t norm_typed(const NormParams &p, int sm_count, cudaStream_t s) {
  const RowShape g = row_shape(p.rows, p.cols, sm_count);
  const int64_t ctas = (p.rows + g.rows - 1) / g.rows;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  const int e = sizeof(T);
  const int vec = (aligned_rows(p.x, p.ldx, e, 16) ? 1 : 0) | (p.r && aligned_rows(p.r, p.ldr, e, 16) ? 2 : 0) |
                  (aligned_rows(p.w, 0, 4, 16) ? 4 : 0) | (p.h && aligned_rows(p.h, p.ldh, e, 16) ? 8 : 0) |
                  (p.y && aligned_rows(p.y, p.ldy, e, 16) ? 16 : 0) | (aligned_rows(p.q, p.ldq, 1, 8) ? 32 : 0);
  const dim3 grid(static_cast<unsigned>(ctas)), block(g.threads, g.rows);
  auto go = [&](auto kernel) { return launch_maybe_pdl(kernel, grid, block, 0, s, true, p, vec); };
  if (g.loop) return go(rms_norm_kernel<T, 4, true>);
  if (g.nv == 1) return go(rms_norm_kernel<T, 1, false>);
  return g.nv == 2 ? go(rms_norm_kernel<T, 2, false>) : go(rms_norm_kernel<T, 4, false>);
}

template <class T>
cudaError_t backward_typed(const NormGradParams &p, int sm_count, cudaStream_t s) {
  RowShape g = row_shape(p.rows, p.cols, sm_count);
  if (g.threads == 32 && g.rows > 1) g = {32, g.nv, 1, false};   // one row at a time a CTA
  const int64_t ctas = p.rows < kNormPartials ? p.rows : kNormPartials;
  const int e = sizeof(T);
  const int vec = (aligned_rows(p.dy, p.lddy, e, 16) ? 1 : 0) | (aligned_rows(p.h, p.ldh, e, 16) ? 2 : 0) |
                  (aligned_rows(p.w, 0, 4, 16) ? 4 : 0) | (p.dh && aligned_rows(p.dh, p.lddh, e, 16) ? 8 : 0) |
                  (aligned_rows(p.dx, p.lddx, e, 16) ? 16 : 0);
  const dim3 grid(static_cast<unsigned>(ctas)), block(g.threads);
  auto go = [&](auto kernel) { return launch_maybe_pdl(kernel, grid, block, 0, s, true, p, vec); };
  if (ctas > 0) {
    const cudaError_t err = g.loop       ? go(rms_norm_backward_kernel<T, 4, true>)
                            : g.nv == 1  ? go(rms_norm_backward_kernel<T, 1, false>)
                            : g.nv == 2  ? go(rms_norm_backward_kernel<T, 2, false>)
                                         : go(rms_norm_backward_kernel<T, 4, false>);
    if (err != cudaSuccess) return err;
  }
  if (!p.dw) return cudaSuccess;
  const dim3 dgrid(static_cast<unsigned>((p.cols + 31) / 32)), dblock(32, 8);
  const int parts = static_cast<int>(ctas);
  if (p.w_f32)
    return launch_maybe_pdl(norm_dw_kernel<float>, dgrid, dblock, 0, s, true, p.partial, parts, p.cols,
                            static_cast<float *>(p.dw));
  return launch_maybe_pdl(norm_dw_kernel<T>, dgrid, dblock, 0, s, true, p.partial, parts, p.cols,
                          static_cast<T *>(p.dw));
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, int sm_count, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return norm_typed<float>(p, sm_count, s);
    case SGEMM_TYPE_BF16: return norm_typed<__nv_bfloat16>(p, sm_count, s);
    default: return norm_typed<__half>(p, sm_count, s);
  }
}

cudaError_t launch_rms_norm_backward(const NormGradParams &p, int sm_count, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return backward_typed<float>(p, sm_count, s);
    case SGEMM_TYPE_BF16: return backward_typed<__nv_bfloat16>(p, sm_count, s);
    default: return backward_typed<__half>(p, sm_count, s);
  }
}

}  // namespace sg
