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
#include <mutex>

#include "dispatch.h"
#include "fp8.cuh"
#include "fp8.h"

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
      // (no correction of the quotient here: y has all its bits, so y / s is seldom in the middle between two 8-bit
      // values; q's error against 64 bits at 8192 x 8192 is 6.1e-4 so, 5.9e-4 with a division, and the registers for
      // the correction cost a third of the resident CTAs, 95 -> 111 us)
      store8_fp8(p.q + row * p.ldq + c, to_fp8x8(y, __fdiv_rn(1.0f, s), p.e5m2), n, vec & 32);
      if ((threadIdx.x & 15) == 0 && n > 0) p.s[row * p.lds + c / 128] = s;
    }
  }
}

// A thread's own 16 bytes from global to its own place in shared memory, asynchronously.
__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most `n` of this thread's groups are in flight.
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

// CTA b takes rows b, b + grid, ... and adds dy h t of its rows per column in registers.  A thread
// copies its own elements of dy, h and dh of the next `depth` rows to places of its own in shared
// memory and reads them there (no barrier but the sum's): bound by memory, it needs some 50 KB in
// flight on every SM, and one row in registers at a time had none during the sum (4095 x 8192 bf16
// 108 us; so, with the sum over rows, 55).
template <class T, int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512, NV == 2 ? 2 : 1)
    rms_norm_backward_kernel(const NormGradParams p, const int vec, const int depth) {
  constexpr int U = sizeof(Raw<T>) / 16;   // 16-byte units of eight elements
  extern __shared__ __align__(16) uint4 rows_smem[];   // [depth][dy, h, dh][NV][U][thread]
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  float dw[NV][8];
  int turn = 0, n[NV];
  const auto column = [&](int j) { return (static_cast<int64_t>(j) * blockDim.x + threadIdx.x) * 8; };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    n[j] = static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - column(j))));
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  }
  const auto place = [&](int slot, int a, int j, int u) {
    return rows_smem + (((slot * 3 + a) * NV + j) * U + u) * blockDim.x + threadIdx.x;
  };
  const auto fetch = [&](int64_t row, int slot) {
    if (row < p.rows) {
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        const T *x = static_cast<const T *>(a == 0 ? p.dy : a == 1 ? p.h : p.dh);
        const int64_t ld = a == 0 ? p.lddy : a == 1 ? p.ldh : p.lddh;
        if (a == 2 && !x) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const T *src = x + row * ld + column(j);
          if (n[j] == 8 && (vec >> a & 1)) {
#pragma unroll
            for (int u = 0; u < U; ++u) copy16(place(slot, a, j, u), reinterpret_cast<const uint4 *>(src) + u);
          } else {
            const Raw<T> r = load8(src, n[j], false);
#pragma unroll
            for (int u = 0; u < U; ++u) *place(slot, a, j, u) = r.u[u];
          }
        }
      }
    }
    copies_commit();
  };
  const auto take = [&](int slot, int a, int j, float (&v)[8]) {
    Raw<T> r;
#pragma unroll
    for (int u = 0; u < U; ++u) r.u[u] = *place(slot, a, j, u);
    unpack(r, v);
  };
  for (int d = 0; d < depth; ++d) fetch(blockIdx.x + static_cast<int64_t>(d) * gridDim.x, d);
  int slot = 0;
  float t_next = p.t[blockIdx.x];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    copies_wait(depth - 1);
    const float t = t_next;
    if (row + gridDim.x < p.rows) t_next = p.t[row + gridDim.x];
    float g[NV][8], sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float d[8], x[8];
      take(slot, 0, j, d);
      take(slot, 1, j, x);
      load_w<T>(p.w, p.w_f32, column(j), n[j], vec & 8, g[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[j][i] *= d[i];
        sum += g[j][i] * x[i];
        dw[j][i] += d[i] * x[i] * t;
      }
    }
    sum = row_sum(sum, red, turn);
    const float k = t * t * (sum / static_cast<float>(p.cols));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8], v[8];
      take(slot, 1, j, x);
      if (p.dh) take(slot, 2, j, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = t * (g[j][i] - x[i] * k);
        v[i] = p.dh ? v[i] + y : y;
      }
      store8(static_cast<T *>(p.dx) + row * p.lddx + column(j), v, n[j], vec & 16);
    }
    fetch(row + static_cast<int64_t>(depth) * gridDim.x, slot);
    slot = slot + 1 == depth ? 0 : slot + 1;
  }
  copies_wait(0);
  if (!p.partial) return;
  const int64_t pitch = (p.cols + 7) / 8 * 8;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (n[j] > 0) store8(p.partial + blockIdx.x * pitch + column(j), dw[j], 8, true);
}

// Rows too long for registers: walked in segments, twice; the sums of dy h t are kept in this CTA's
// row of the workspace.
template <class T>
__global__ void __launch_bounds__(512) rms_norm_backward_long_kernel(const NormGradParams p, const int vec) {
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t pitch = (p.cols + 7) / 8 * 8, step = static_cast<int64_t>(8) * blockDim.x;
  int turn = 0;
  float dy[8], h[8], w[8];
  const auto load = [&](int64_t row, int64_t c) {
    const int n = static_cast<int>(min(int64_t(8), p.cols - c));
    unpack(load8(static_cast<const T *>(p.dy) + row * p.lddy + c, n, vec & 1), dy);
    unpack(load8(static_cast<const T *>(p.h) + row * p.ldh + c, n, vec & 2), h);
    load_w<T>(p.w, p.w_f32, c, n, vec & 8, w);
    return n;
  };
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float t = p.t[row];
    float sum = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += step) {
      load(row, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += dy[i] * w[i] * h[i];
    }
    sum = row_sum(sum, red, turn);
    const float k = t * t * (sum / static_cast<float>(p.cols));
    for (int64_t c = threadIdx.x * 8; c < p.cols; c += step) {
      const int n = load(row, c);
      float v[8];
      if (p.dh) unpack(load8(static_cast<const T *>(p.dh) + row * p.lddh + c, n, vec & 4), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = t * (dy[i] * w[i] - h[i] * k);
        v[i] = p.dh ? v[i] + d : d;
      }
      store8(static_cast<T *>(p.dx) + row * p.lddx + c, v, n, vec & 16);
      if (p.partial) {   // no other thread touches these
        float *mine = p.partial + blockIdx.x * pitch + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[i] = (row == blockIdx.x ? 0.0f : mine[i]) + dy[i] * h[i] * t;
      }
    }
  }
}

// dw[c] = sum over the CTAs' partial rows, in a fixed order: every 32nd of them by one thread (ten
// loads in flight), then the 32 sums.
template <class T>
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *partial, int parts, int64_t cols, T *dw) {
  __shared__ float red[32][33];
  griddep_wait();
  const int64_t pitch = (cols + 7) / 8 * 8;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float sum = 0.0f;
  for (int r0 = threadIdx.y; r0 < parts; r0 += 320) {
    float v[10];
#pragma unroll
    for (int i = 0; i < 10; ++i) v[i] = c < cols && r0 + 32 * i < parts ? partial[(r0 + 32 * i) * pitch + c] : 0.0f;
#pragma unroll
    for (int i = 0; i < 10; ++i) sum += v[i];
  }
  red[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  sum = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < cols) from_float(dw + o, sum);
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

// The backward kernel's threads and chunks a thread, and the CTAs that share an SM (about 1024 threads;
// the 4-chunk form's registers allow one).
struct GradShape {
  int threads, nv, per_sm;
};
GradShape grad_shape(int64_t cols, int elem) {
  const int64_t chunks = (cols + 7) / 8;
  GradShape g = {512, 0, 2};   // nv 0: rows longer than the registers hold
  if (chunks <= 256 || (elem == 4 && chunks <= 1024))
    g = {static_cast<int>((chunks + 31) / 32 * 32), 1, 0};
  else if (chunks <= 1024)
    g = {static_cast<int>(((chunks + 1) / 2 + 31) / 32 * 32), 2, 0};
  else if (chunks <= 2048)
    return {static_cast<int>(((chunks + 3) / 4 + 31) / 32 * 32), 4, 1};
  if (g.nv > 0) g.per_sm = 1024 / g.threads < 8 ? (1024 / g.threads > 1 ? 1024 / g.threads : 1) : 8;
  return g;
}
constexpr int kSms = 152;   // of a GB300: sizes the partial sums, whose number must not depend on the device
int64_t grad_ctas(int64_t rows, const GradShape &g) {
  const int64_t most = static_cast<int64_t>(kSms) * g.per_sm;
  return rows < most ? rows : most;
}

// Rows in flight per CTA: up to four, as far as the CTAs of an SM find room in its shared memory.
template <class T, int NV>
cudaError_t launch_backward(const NormGradParams &p, const GradShape &g, int vec, cudaStream_t s) {
  const int row_bytes = 3 * NV * g.threads * static_cast<int>(sizeof(Raw<T>));
  const int fit = 224 * 1024 / g.per_sm / row_bytes;
  const int depth = fit < 1 ? 1 : fit < 4 ? fit : 4;
  static std::once_flag once[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [] {
    cudaFuncSetAttribute(rms_norm_backward_kernel<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
  });
  return launch_maybe_pdl(rms_norm_backward_kernel<T, NV>, dim3(static_cast<unsigned>(grad_ctas(p.rows, g))),
                          dim3(g.threads), static_cast<size_t>(depth) * row_bytes, s, true, p, vec, depth);
}

template <class T>
cudaError_t backward_typed(const NormGradParams &p, cudaStream_t s) {
  const GradShape g = grad_shape(p.cols, sizeof(T));
  const int64_t ctas = grad_ctas(p.rows, g);
  const int e = sizeof(T);
  const int vec = (aligned_rows(p.dy, p.lddy, e, 16) ? 1 : 0) | (aligned_rows(p.h, p.ldh, e, 16) ? 2 : 0) |
                  (p.dh && aligned_rows(p.dh, p.lddh, e, 16) ? 4 : 0) | (aligned_rows(p.w, 0, 4, 16) ? 8 : 0) |
                  (aligned_rows(p.dx, p.lddx, e, 16) ? 16 : 0);
  if (ctas > 0) {
    cudaError_t err;
    if constexpr (sizeof(T) == 4) {   // two chunks a thread: 16-bit rows only
      err = cudaErrorInvalidConfiguration;
    } else {
      if (g.nv == 2) err = launch_backward<T, 2>(p, g, vec, s);
    }
    if (g.nv == 1) err = launch_backward<T, 1>(p, g, vec, s);
    if (g.nv == 4) err = launch_backward<T, 4>(p, g, vec, s);
    if (g.nv == 0)
      err = launch_maybe_pdl(rms_norm_backward_long_kernel<T>, dim3(static_cast<unsigned>(ctas)), dim3(g.threads), 0, s,
                             true, p, vec);
    if (err != cudaSuccess) return err;
  }
  if (!p.dw) return cudaSuccess;
  const dim3 dgrid(static_cast<unsigned>((p.cols + 31) / 32)), dblock(32, 32);
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

int64_t norm_partials(int64_t rows, int64_t cols) {
  const int64_t a = grad_ctas(rows, grad_shape(cols, 2)), b = grad_ctas(rows, grad_shape(cols, 4));
  return a > b ? a : b;
}

cudaError_t launch_rms_norm_backward(const NormGradParams &p, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return backward_typed<float>(p, s);
    case SGEMM_TYPE_BF16: return backward_typed<__nv_bfloat16>(p, s);
    default: return backward_typed<__half>(p, s);
  }
}

}  // namespace sg
