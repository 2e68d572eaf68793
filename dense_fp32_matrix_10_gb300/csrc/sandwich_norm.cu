// sandwich_norm.cu -- the norm behind a block, its gate, the scaled residual
// and the norm in front of the next block, with a quantised output, and their
// gradient.
//
//   tp = 1 / sqrt(mean a^2 + eps),  h = rho x + gate (a tp wp)
//   t  = 1 / sqrt(mean h^2 + eps),  y = h t w,  (q, s) = y in 1 x 128 blocks
//
//   H  = t (dy w - h t^2 mean(dy w h)) + dh,  dx = rho H
//   v  = H gate wp,  da = tp (v - a tp^2 mean(v a))
//   dw = sum dy h t,  dwp = sum H gate a tp,  dgate = wp sum H a tp
//
// The gradient's second mean is that of a sum which is linear in the first,
// so both come from three sums over the row, taken together:
//   A = sum dy w h,  P = sum (t dy w + dh) p,  R = sum h p   with p = gate wp a
//   sum v a = P - t^3 (A / cols) R
#include <mutex>

#include "dispatch.h"
#include "fp8_block.cuh"
#include "row_norm.cuh"

namespace sg {
namespace {

// vec: bit 0 a, 1 x, 2 w, 3 wp, 4 gate, 5 h (16-byte rows), 6 q, 7 qa, 8 qh (8-byte rows)
template <class T, int NV, bool LONG>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) sandwich_norm_kernel(const SandwichParams p, const int vec) {
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;   // whole warps: a CTA of several warps per row has blockDim.y == 1
  const T *a = static_cast<const T *>(p.a) + row * p.lda, *x = static_cast<const T *>(p.x) + row * p.ldx;
  const int64_t gate_row = p.gate.p ? static_cast<unsigned>(row) / p.gate.rows * p.gate.ld : 0;
  const int64_t seg = static_cast<int64_t>(8) * NV * blockDim.x;
  int turn = 0;
  float va[NV][8], h[NV][8];
  const auto column = [&](int64_t base, int j) { return base + (static_cast<int64_t>(j) * blockDim.x + threadIdx.x) * 8; };
  const auto count = [&](int64_t c) { return static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c))); };
  const auto load_a = [&](int64_t base) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = column(base, j);
      unpack(load8(a + c, count(c), vec & 1), va[j]);
    }
  };
  Raw<T> rx[NV];
  const auto load_x = [&](int64_t base) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = column(base, j);
      rx[j] = load8(x + c, count(c), vec & 2);
    }
  };
  // h of a segment from its a and x
  const auto make_h = [&](int64_t base, float tp) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = column(base, j);
      const int n = count(c);
      float wp[8], gate[8];
      unpack(rx[j], h[j]);
      load_w<T>(p.wp, p.w_f32, c, n, vec & 8, wp);
      if (p.gate.p) load_w<T>(p.gate.p, p.gate.f32, gate_row + c, n, vec & 16, gate);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float u = va[j][i] * tp * wp[i];
        if (p.gate.p) u *= gate[i];
        h[j][i] = i < n ? fmaf(p.residual_scale, h[j][i], u) : 0.0f;
      }
    }
  };
  const int64_t end = LONG ? p.cols : 1;
  load_a(0);
  load_x(0);
  float sum = 0.0f;
  for (int64_t base = 0; base < end; base += seg) {
    if (LONG) load_a(base);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += va[j][i] * va[j][i];
  }
  sum = row_sum(sum, red, turn);
  const float tp = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  if (p.tp && threadIdx.x == 0) p.tp[row] = tp;
  sum = 0.0f;
  for (int64_t base = 0; base < end; base += seg) {
    if (LONG) {
      load_a(base);
      load_x(base);
    }
    make_h(base, tp);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += h[j][i] * h[j][i];
  }
  sum = row_sum(sum, red, turn);
  const float t = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
  if (p.t && threadIdx.x == 0) p.t[row] = t;
  for (int64_t base = 0; base < end; base += seg) {
    if (LONG) {
      load_a(base);
      load_x(base);
      make_h(base, tp);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = column(base, j);
      const int n = count(c);
      store8(static_cast<T *>(p.h) + row * p.ldh + c, h[j], n, vec & 32);
      if (p.qa) store_block(va[j], n, p.qa + row * p.ldqa + c, p.sa + row * p.ldsa + c / 128, p.keep_e5m2, vec & 128);
      if (p.qh) store_block(h[j], n, p.qh + row * p.ldqh + c, p.sh + row * p.ldsh + c / 128, p.keep_e5m2, vec & 256);
      float w[8], y[8];
      load_w<T>(p.w, p.w_f32, c, n, vec & 4, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[j][i] * t * w[i];
      store_block(y, n, p.q + row * p.ldq + c, p.s + row * p.lds + c / 128, p.e5m2, vec & 64);
    }
  }
}

// ------------------------------------------------------------------ gradient
// The workspace: for every CTA a row of `pitch` floats for each of dw, dwp,
// and dgate's sums over the rows of the first and of the last gate row that it
// shares with other CTAs.
enum : int { kDw = 0, kDwp = 1, kHead = 2, kTail = 3, kParts = 4 };

// CTAs, each with `rows` consecutive rows (the last one fewer).
struct Split {
  unsigned ctas, rows;
};

__device__ __forceinline__ float *part(float *partial, int64_t pitch, unsigned cta, int kind) {
  return partial + (static_cast<int64_t>(cta) * kParts + kind) * pitch;
}

template <class T>
__device__ __forceinline__ void load_kept(const Kept &k, int64_t row, int64_t c, int n, bool vec, float (&v)[8]) {
  if (k.s) {
    unpack_fp8(load8_fp8(static_cast<const unsigned char *>(k.p) + row * k.ld + c, n, vec), k.e5m2, v);
    const float s = n > 0 ? k.s[row * k.lds + c / 128] : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] * s : 0.0f;
  } else {
    unpack(load8(static_cast<const T *>(k.p) + row * k.ld + c, n, vec), v);
  }
}
template <class T>
__device__ __forceinline__ void store_w(void *w, bool f32, int64_t c, const float (&v)[8], int n) {
  if (f32)
    store8(static_cast<float *>(w) + c, v, n, false);
  else
    store8(static_cast<T *>(w) + c, v, n, false);
}

// row_sum() of three values.
__device__ __forceinline__ void row_sums(float &a, float &b, float &c, float (*red)[3][32], int &turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  c = warp_sum(c);
  if (blockDim.x == 32) return;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    red[turn][0][threadIdx.x >> 5] = a;
    red[turn][1][threadIdx.x >> 5] = b;
    red[turn][2][threadIdx.x >> 5] = c;
  }
  __syncthreads();
  a = warp_sum(lane < warps ? red[turn][0][lane] : 0.0f);
  b = warp_sum(lane < warps ? red[turn][1][lane] : 0.0f);
  c = warp_sum(lane < warps ? red[turn][2][lane] : 0.0f);
  turn ^= 1;
}

// vec: bit 0 dy, 1 dh, 2 w, 3 wp, 4 gate, 5 da, 6 dx (16-byte rows), 7 a, 8 h (16, or 8 of checkpoints)
template <class T, int NV, bool LONG>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) sandwich_backward_kernel(const SandwichGradParams p,
                                                                                 const Split split, const int vec) {
  __shared__ float red[2][3][32];
  griddep_wait();
  griddep_launch_dependents();
  const unsigned r0 = blockIdx.x * split.rows;
  const unsigned r1 = static_cast<unsigned>(min(static_cast<int64_t>(r0) + split.rows, p.rows));
  const int64_t pitch = (p.cols + 7) / 8 * 8, seg = static_cast<int64_t>(8) * NV * blockDim.x;
  const int64_t end = LONG ? p.cols : 1;
  const float mean = 1.0f / static_cast<float>(p.cols);
  int turn = 0;
  // sums over rows: of this thread's columns, or (LONG) in this CTA's rows of the workspace, the running sum of
  // H a tp in its head row
  float sw[NV][8], swp[NV][8], sn[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) sw[j][i] = swp[j][i] = sn[j][i] = 0.0f;
  const auto column = [&](int64_t base, int j) { return base + (static_cast<int64_t>(j) * blockDim.x + threadIdx.x) * 8; };
  const auto count = [&](int64_t c) { return static_cast<int>(max(int64_t(0), min(int64_t(8), p.cols - c))); };
  float dy[NV][8], h[NV][8], a[NV][8], dh[NV][8];
  const auto load = [&](int64_t row, int64_t base) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t c = column(base, j);
      const int n = count(c);
      unpack(load8(static_cast<const T *>(p.dy) + row * p.lddy + c, n, vec & 1), dy[j]);
      load_kept<T>(p.h, row, c, n, vec & 256, h[j]);
      load_kept<T>(p.a, row, c, n, vec & 128, a[j]);
      if (p.dh) {
        unpack(load8(static_cast<const T *>(p.dh) + row * p.lddh + c, n, vec & 2), dh[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) dh[j][i] = 0.0f;
      }
    }
  };
  for (unsigned row = r0; row < r1; ++row) {
    const float t = p.t[row], tp = p.tp[row];
    const unsigned group = p.gate.p ? row / p.gate.rows : 0;
    const int64_t gate_row = group * p.gate.ld;
    float A = 0.0f, P = 0.0f, R = 0.0f;
    for (int64_t base = 0; base < end; base += seg) {
      load(row, base);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t c = column(base, j);
        const int n = count(c);
        float w[8], wp[8], gate[8];
        load_w<T>(p.w, p.w_f32, c, n, vec & 4, w);
        load_w<T>(p.wp, p.w_f32, c, n, vec & 8, wp);
        if (p.gate.p) load_w<T>(p.gate.p, p.gate.f32, gate_row + c, n, vec & 16, gate);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = dy[j][i] * w[i], q = a[j][i] * (p.gate.p ? gate[i] * wp[i] : wp[i]);
          A += g * h[j][i];
          P += (t * g + dh[j][i]) * q;
          R += h[j][i] * q;
        }
      }
    }
    row_sums(A, P, R, red, turn);
    const float k = t * t * (A * mean);            // H = t (g - h k) + dh
    const float kp = tp * tp * ((P - t * k * R) * mean);   // da = tp (v - a kp)
    for (int64_t base = 0; base < end; base += seg) {
      if (LONG) load(row, base);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int64_t c = column(base, j);
        const int n = count(c);
        float w[8], wp[8], gate[8], dx[8], da[8];
        load_w<T>(p.w, p.w_f32, c, n, vec & 4, w);
        load_w<T>(p.wp, p.w_f32, c, n, vec & 8, wp);
        if (p.gate.p) load_w<T>(p.gate.p, p.gate.f32, gate_row + c, n, vec & 16, gate);
        if (LONG) {
          // (no other thread touches these)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool old = p.partial && n > 0 && row != r0;
            sw[j][i] = old ? part(p.partial, pitch, blockIdx.x, kDw)[c + i] : 0.0f;
            swp[j][i] = old ? part(p.partial, pitch, blockIdx.x, kDwp)[c + i] : 0.0f;
            sn[j][i] = old && !(p.gate.p && row % p.gate.rows == 0) ? part(p.partial, pitch, blockIdx.x, kTail)[c + i] : 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float H = t * (dy[j][i] * w[i] - h[j][i] * k) + dh[j][i];
          const float v = H * (p.gate.p ? gate[i] * wp[i] : wp[i]);
          dx[i] = p.residual_scale * H;
          da[i] = tp * (v - a[j][i] * kp);
          sw[j][i] += dy[j][i] * h[j][i] * t;
          sn[j][i] += H * a[j][i] * tp;
        }
        store8(static_cast<T *>(p.da) + row * p.ldda + c, da, n, vec & 32);
        store8(static_cast<T *>(p.dx) + row * p.lddx + c, dx, n, vec & 64);
        if (!p.partial || n <= 0) continue;
        // the end of this CTA's rows of a gate row
        bool flush = row + 1 == r1;
        if (p.gate.p) {
          const int64_t g0 = static_cast<int64_t>(group) * p.gate.rows, g1 = min(g0 + p.gate.rows, p.rows);
          flush |= row + 1 == g1;
          if (flush) {
#pragma unroll
            for (int i = 0; i < 8; ++i) swp[j][i] += gate[i] * sn[j][i];
            if (p.dgate) {
              if (g0 >= r0 && g1 <= r1) {
                float dg[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) dg[i] = wp[i] * sn[j][i];
                store_w<T>(p.dgate, p.gate.f32, group * p.lddgate + c, dg, n);
              } else {
                store8(part(p.partial, pitch, blockIdx.x, g0 < r0 ? kHead : kTail) + c, sn[j], 8, true);
              }
            }
          }
        } else if (flush) {
#pragma unroll
          for (int i = 0; i < 8; ++i) swp[j][i] += sn[j][i];
        }
        if (LONG || row + 1 == r1) {
          store8(part(p.partial, pitch, blockIdx.x, kDw) + c, sw[j], 8, true);
          store8(part(p.partial, pitch, blockIdx.x, kDwp) + c, swp[j], 8, true);
          if (LONG && !flush) store8(part(p.partial, pitch, blockIdx.x, kTail) + c, sn[j], 8, true);
        }
        if (flush) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sn[j][i] = 0.0f;
        }
      }
    }
  }
}

// Sums over CTAs in a fixed order: blockIdx.y 0 of dw, 1 of dwp, then of the gate rows that several CTAs share, which
// are found by the gate row (by_group) or by the boundary between two CTAs.
template <class T>
__global__ void __launch_bounds__(1024) sandwich_sums_kernel(const SandwichGradParams p, const Split split,
                                                             const bool by_group) {
  __shared__ float red[32][33];
  griddep_wait();
  const int64_t pitch = (p.cols + 7) / 8 * 8, c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  unsigned first = 0, end = split.ctas, group = 0;
  if (blockIdx.y >= 2) {
    group = blockIdx.y - 2;
    if (!by_group) {
      const int64_t boundary = static_cast<int64_t>(blockIdx.y - 1) * split.rows;
      group = static_cast<unsigned>(boundary / p.gate.rows);
      // the first boundary inside it only
      const int64_t g0 = static_cast<int64_t>(group) * p.gate.rows;
      if (g0 == boundary || g0 < boundary - split.rows) return;
    }
    const int64_t g0 = static_cast<int64_t>(group) * p.gate.rows, g1 = min(g0 + p.gate.rows, p.rows);
    first = static_cast<unsigned>(g0 / split.rows);
    end = static_cast<unsigned>((g1 - 1) / split.rows) + 1;
    if (first + 1 == end) return;
  } else if (!(blockIdx.y ? p.dwp : p.dw)) {
    return;
  }
  float sum = 0.0f;
  for (unsigned b = first + threadIdx.y; b < end; b += 32) {
    const int kind = blockIdx.y == 0 ? kDw : blockIdx.y == 1 ? kDwp : static_cast<int64_t>(group) * p.gate.rows <
                                                                          static_cast<int64_t>(b) * split.rows ? kHead : kTail;
    if (c < p.cols) sum += part(p.partial, pitch, b, kind)[c];
  }
  red[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  sum = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x != 0 || o >= p.cols) return;
  if (blockIdx.y < 2) {
    void *d = blockIdx.y ? p.dwp : p.dw;
    if (p.w_f32)
      static_cast<float *>(d)[o] = sum;
    else
      from_float(static_cast<T *>(d) + o, sum);
  } else {
    sum *= p.w_f32 ? static_cast<const float *>(p.wp)[o] : to_float(static_cast<const T *>(p.wp)[o]);
    if (p.gate.f32)
      static_cast<float *>(p.dgate)[group * p.lddgate + o] = sum;
    else
      from_float(static_cast<T *>(p.dgate) + group * p.lddgate + o, sum);
  }
}

template <class T>
cudaError_t forward_typed(const SandwichParams &p, int sm_count, cudaStream_t s) {
  const RowShape g = row_shape(p.rows, p.cols, sm_count);
  const int64_t ctas = (p.rows + g.rows - 1) / g.rows;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  const int e = sizeof(T), ew = p.w_f32 ? 4 : e, eg = p.gate.f32 ? 4 : e;
  const int vec = (aligned_rows(p.a, p.lda, e, 16) ? 1 : 0) | (aligned_rows(p.x, p.ldx, e, 16) ? 2 : 0) |
                  (aligned_rows(p.w, 0, ew, 16) ? 4 : 0) | (aligned_rows(p.wp, 0, ew, 16) ? 8 : 0) |
                  (aligned_rows(p.gate.p, p.gate.ld, eg, 16) ? 16 : 0) | (aligned_rows(p.h, p.ldh, e, 16) ? 32 : 0) |
                  (aligned_rows(p.q, p.ldq, 1, 8) ? 64 : 0) | (aligned_rows(p.qa, p.ldqa, 1, 8) ? 128 : 0) |
                  (aligned_rows(p.qh, p.ldqh, 1, 8) ? 256 : 0);
  const dim3 grid(static_cast<unsigned>(ctas)), block(g.threads, g.rows);
  auto go = [&](auto kernel) { return launch_maybe_pdl(kernel, grid, block, 0, s, true, p, vec); };
  if (g.loop) return go(sandwich_norm_kernel<T, 4, true>);
  if (g.nv == 1) return go(sandwich_norm_kernel<T, 1, false>);
  return g.nv == 2 ? go(sandwich_norm_kernel<T, 2, false>) : go(sandwich_norm_kernel<T, 4, false>);
}

// Threads and chunks a thread of the gradient, and the CTAs of its grid (a number that does not depend on the device).
struct GradShape {
  int threads, nv;
  bool loop;
  Split split;
};
GradShape grad_shape(int64_t rows, int64_t cols) {
  const int64_t chunks = (cols + 7) / 8;
  auto up32 = [](int64_t v) { return static_cast<int>((v + 31) / 32 * 32); };
  GradShape g = {512, 1, true, {}};
  if (chunks <= 512)
    g = {up32(chunks), 1, false, {}};
  else if (chunks <= 1024)
    g = {up32((chunks + 1) / 2), 2, false, {}};
  const int64_t most = 152 * (g.threads >= 1024 ? 1 : 1024 / g.threads < 8 ? 1024 / g.threads : 8);
  g.split.rows = rows > 0 ? static_cast<unsigned>((rows + most - 1) / most) : 1;
  g.split.ctas = static_cast<unsigned>((rows + g.split.rows - 1) / g.split.rows);
  return g;
}

template <class T>
cudaError_t backward_typed(const SandwichGradParams &p, cudaStream_t s, int *launches) {
  const bool sums = p.dw || p.dwp || p.dgate;
  const GradShape g = grad_shape(p.rows, p.cols);
  const int e = sizeof(T), ew = p.w_f32 ? 4 : e, eg = p.gate.f32 ? 4 : e;
  const auto kept = [&](const Kept &k) { return k.s ? aligned_rows(k.p, k.ld, 1, 8) : aligned_rows(k.p, k.ld, e, 16); };
  const int vec = (aligned_rows(p.dy, p.lddy, e, 16) ? 1 : 0) | (aligned_rows(p.dh, p.lddh, e, 16) ? 2 : 0) |
                  (aligned_rows(p.w, 0, ew, 16) ? 4 : 0) | (aligned_rows(p.wp, 0, ew, 16) ? 8 : 0) |
                  (aligned_rows(p.gate.p, p.gate.ld, eg, 16) ? 16 : 0) | (aligned_rows(p.da, p.ldda, e, 16) ? 32 : 0) |
                  (aligned_rows(p.dx, p.lddx, e, 16) ? 64 : 0) | (kept(p.a) ? 128 : 0) | (kept(p.h) ? 256 : 0);
  const dim3 grid(g.split.ctas), block(g.threads);
  auto go = [&](auto kernel) { return launch_maybe_pdl(kernel, grid, block, 0, s, true, p, g.split, vec); };
  if (p.rows > 0) {
    const cudaError_t err = g.loop      ? go(sandwich_backward_kernel<T, 1, true>)
                            : g.nv == 1 ? go(sandwich_backward_kernel<T, 1, false>)
                                        : go(sandwich_backward_kernel<T, 2, false>);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  if (!sums) return cudaSuccess;
  unsigned shared = 0;   // gate rows to be looked at
  bool by_group = false;
  if (p.dgate && p.rows > 0 && g.split.rows % p.gate.rows != 0) {
    const int64_t groups = (p.rows + p.gate.rows - 1) / p.gate.rows;
    by_group = groups < g.split.ctas;
    shared = by_group ? static_cast<unsigned>(groups) : g.split.ctas - 1;
  }
  ++*launches;
  return launch_maybe_pdl(sandwich_sums_kernel<T>, dim3(static_cast<unsigned>((p.cols + 31) / 32), 2 + shared),
                          dim3(32, 32), 0, s, true, p, g.split, by_group);
}

}  // namespace

cudaError_t launch_sandwich_norm(const SandwichParams &p, int sm_count, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return forward_typed<float>(p, sm_count, s);
    case SGEMM_TYPE_BF16: return forward_typed<__nv_bfloat16>(p, sm_count, s);
    default: return forward_typed<__half>(p, sm_count, s);
  }
}

int64_t sandwich_partials(int64_t rows, int64_t cols) {
  return static_cast<int64_t>(grad_shape(rows, cols).split.ctas) * kParts * ((cols + 7) / 8 * 8);
}

cudaError_t launch_sandwich_norm_backward(const SandwichGradParams &p, cudaStream_t s, int *launches) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return backward_typed<float>(p, s, launches);
    case SGEMM_TYPE_BF16: return backward_typed<__nv_bfloat16>(p, s, launches);
    default: return backward_typed<__half>(p, s, launches);
  }
}

}  // namespace sg
