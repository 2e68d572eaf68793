// sandwich_backward.cu -- the gradient of the norms around a block
// (sandwich_norm.cuh has the formulas).
//
// The second mean is that of a sum which is linear in the first, so both come
// from three sums over the row, taken together:
//   A = sum dy w h,  P = sum (t dy w + dh) p,  R = sum h p   with p = gate wp a
//   sum v a = P - t^3 (A / cols) R
#include "sandwich_norm.cuh"

namespace sg {
namespace {

constexpr int kSms = 152;   // of a GB300: sizes the partial sums, whose number must not depend on the device

// The workspace: for every CTA a row of `pitch` floats for each of dw, dwp, and dgate's sums over the rows of the first
// and of the last gate row that it shares with other CTAs.
enum : int { kDw = 0, kDwp = 1, kHead = 2, kTail = 3, kParts = 4 };
inline __host__ __device__ int64_t part_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }
__device__ __forceinline__ float *part(const SandwichGradParams &p, unsigned cta, int kind, int64_t c) {
  return p.partial + (static_cast<int64_t>(cta) * kParts + kind) * part_pitch(p.cols) + c;
}
__device__ __forceinline__ void load_part(const float *at, float2 (&v)[8]) { unpack(load16(at, 16, 1), v); }
__device__ __forceinline__ void store_part(float *at, const float2 (&v)[8]) { store16(at, v, 16, 1); }

// What a row's sums over rows add up to at the end of a CTA's rows of a gate row (`group`, whose gate wp m goes with): its
// part of dwp is added to the CTA's, and its part of dgate is stored, or dgate itself if all its rows are this CTA's.
template <class T>
__device__ __forceinline__ void flush(const SandwichGradParams &p, unsigned group, unsigned r0, unsigned r1, int64_t c, int n,
                                      const float2 (&sn)[8], bool first, uint32_t vec) {
  float2 v[8];
  if (p.gate.p) {
    load16_w<T>(p.gate.p, p.gate.f32, group * p.gate.ld + c, n, level(vec, 4), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], sn[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sn[i];
  }
  float *dwp = part(p, blockIdx.x, kDwp, c);
  if (!first) {
    float2 old[8];
    load_part(dwp, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = add2(v[i], old[i]);
  }
  store_part(dwp, v);
  if (!p.dgate) return;
  const int64_t g0 = static_cast<int64_t>(group) * p.gate.rows, g1 = min(g0 + p.gate.rows, p.rows);
  if (g0 >= r0 && g1 <= r1) {
    load16_w<T>(p.wp, p.w_f32, c, n, level(vec, 3), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], sn[i]);
    const int64_t at = group * p.lddgate + c;
    if (p.gate.f32)
      store16(static_cast<float *>(p.dgate) + at, v, n, level(vec, 9));
    else
      store16(static_cast<T *>(p.dgate) + at, v, n, level(vec, 9));
  } else {
    store_part(part(p, blockIdx.x, g0 < r0 ? kHead : kTail, c), sn);
  }
}

template <class T>
__device__ __forceinline__ void load_gated(const SandwichGradParams &p, unsigned group, int64_t c, int n, uint32_t vec,
                                           float2 (&m)[8]) {
  load16_w<T>(p.wp, p.w_f32, c, n, level(vec, 3), m);
  if (p.gate.p) {
    float2 g[8];
    load16_w<T>(p.gate.p, p.gate.f32, group * p.gate.ld + c, n, level(vec, 4), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = mul2(m[i], g[i]);
  }
}
__device__ __forceinline__ void unpack_kept(uint4 u, float scale, bool e5m2, float2 (&v)[8]) {
  if (e5m2)
    unpack_fp8<true>(u, v);
  else
    unpack_fp8<false>(u, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], both(scale));
}

// Sixteen elements of a row's inputs.
struct Inputs {
  float2 dy[8], dh[8], a[8], h[8];
};
// A, P and R over them.
__device__ __forceinline__ void add_sums(const Inputs &x, const float2 (&w)[8], const float2 (&m)[8], float t, float &A,
                                         float &P, float &R) {
  float2 sa = both(0.0f), sp = both(0.0f), sr = both(0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 g = mul2(x.dy[i], w[i]), q = mul2(x.a[i], m[i]);
    sa = fma2(g, x.h[i], sa);
    sp = fma2(fma2(both(t), g, x.dh[i]), q, sp);
    sr = fma2(x.h[i], q, sr);
  }
  A += sa.x + sa.y;
  P += sp.x + sp.y;
  R += sr.x + sr.y;
}
// The factors of a row: H = t g - th h + dh, da = tp v - tpa a.
struct Factors {
  float t, tp, th, tpa;
};
__device__ __forceinline__ Factors factors(float t, float tp, float A, float P, float R, float mean) {
  const float th = t * (t * t * (A * mean));
  return {t, tp, th, tp * (tp * tp * ((P - th * R) * mean))};
}
template <class T>
__device__ __forceinline__ void finish(const SandwichGradParams &p, int64_t row, int64_t c, int n, const Inputs &x,
                                       const float2 (&w)[8], const float2 (&m)[8], const Factors &f, float2 (&sw)[8],
                                       float2 (&sn)[8], uint32_t vec) {
  float2 da[8], dx[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 H = fma2(both(f.t), mul2(x.dy[i], w[i]), fma2(both(-f.th), x.h[i], x.dh[i]));
    da[i] = fma2(both(f.tp), mul2(H, m[i]), mul2(both(-f.tpa), x.a[i]));
    dx[i] = mul2(both(p.residual_scale), H);
    sw[i] = fma2(mul2(x.dy[i], both(f.t)), x.h[i], sw[i]);
    sn[i] = fma2(H, mul2(x.a[i], both(f.tp)), sn[i]);
  }
  store16(static_cast<T *>(p.da) + row * p.ldda + c, da, n, level(vec, 5));
  store16(static_cast<T *>(p.dx) + row * p.lddx + c, dx, n, level(vec, 6));
}

// KA, KH: a and h are checkpoints.  vec: 0 dy, 1 dh, 2 w, 3 wp, 4 gate, 5 da, 6 dx, 7 a, 8 h, 9 dgate
template <class T, bool KA, bool KH>
struct RowPlaces {
  static constexpr int U = sizeof(T), kDh = U, kA = 2 * U, kH = kA + (KA ? 1 : U), kUnits = kH + (KH ? 1 : U);
  static constexpr int kScales = (KA ? 1 : 0) + (KH ? 1 : 0), kBytes = kUnits * 16 + kScales * 4;   // of a thread
};
template <class T, bool KA, bool KH>
__global__ void __launch_bounds__(kRowThreads, 1) sandwich_backward_kernel(const SandwichGradParams p, const Split split,
                                                                           const int depth, const uint32_t vec) {
  using At = RowPlaces<T, KA, KH>;
  extern __shared__ __align__(16) uint4 rows_smem[];   // [depth][dy, dh, a, h][thread], then [depth][scales of checkpoints][thread]
  __shared__ float red[2][4][16];
  griddep_wait();
  griddep_launch_dependents();
  const int step = blockDim.x;
  const unsigned r0 = blockIdx.x * split.rows;
  const unsigned r1 = static_cast<unsigned>(min(static_cast<int64_t>(r0) + split.rows, p.rows));
  const int64_t c = threadIdx.x * 16;
  const int n = static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - c)));
  uint4 *mine = rows_smem + threadIdx.x;
  float *scales = reinterpret_cast<float *>(rows_smem + depth * At::kUnits * step) + threadIdx.x;
  const auto fetch = [&](unsigned row, int slot) {
    if (row < r1) {
      uint4 *to = mine + slot * At::kUnits * step;
      float *s = scales + slot * At::kScales * step;
      copy16(to, step, static_cast<const T *>(p.dy) + row * p.lddy + c, n, level(vec, 0));
      if (p.dh) copy16(to + At::kDh * step, step, static_cast<const T *>(p.dh) + row * p.lddh + c, n, level(vec, 1));
      const auto matrix = [&](const Kept &k, bool kept, int lv, uint4 *place, float *scale) {
        if (kept)
          copy16_kept(place, scale, static_cast<const unsigned char *>(k.p) + row * k.ld + c, k.s + row * k.lds + (c >> 7), n, lv);
        else
          copy16(place, step, static_cast<const T *>(k.p) + row * k.ld + c, n, lv);
      };
      matrix(p.a, KA, level(vec, 7), to + At::kA * step, s);
      matrix(p.h, KH, level(vec, 8), to + At::kH * step, s + (KA ? step : 0));
    }
    copies_commit();
  };
  const auto take = [&](int slot, Inputs &x) {
    const uint4 *at = mine + slot * At::kUnits * step;
    const float *s = scales + slot * At::kScales * step;
    unpack(take16<T>(at, step), x.dy);
    if (p.dh) {
      unpack(take16<T>(at + At::kDh * step, step), x.dh);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.dh[i] = both(0.0f);
    }
    if constexpr (KA)
      unpack_kept(at[At::kA * step], s[0], p.a.e5m2, x.a);
    else
      unpack(take16<T>(at + At::kA * step, step), x.a);
    if constexpr (KH)
      unpack_kept(at[At::kH * step], s[KA ? step : 0], p.h.e5m2, x.h);
    else
      unpack(take16<T>(at + At::kH * step, step), x.h);
  };
  for (int d = 0; d < depth; ++d) fetch(r0 + d, d);
  float2 w[8], m[8], sw[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sw[i] = sn[i] = both(0.0f);
  load16_w<T>(p.w, p.w_f32, c, n, level(vec, 2), w);
  unsigned group = p.gate.p ? r0 / p.gate.rows : 0, group_end = p.gate.p ? (group + 1) * p.gate.rows : ~0u;
  load_gated<T>(p, group, c, n, vec, m);
  const float mean = 1.0f / static_cast<float>(p.cols);
  int turn = 0, slot = 0;
  bool first = true;
  float t_next = p.t[r0], tp_next = p.tp[r0];
  for (unsigned row = r0; row < r1; ++row) {
    if (row >= group_end) {
      ++group;
      group_end += p.gate.rows;
      load_gated<T>(p, group, c, n, vec, m);
    }
    copies_wait(depth - 1);
    const float t = t_next, tp = tp_next;
    if (row + 1 < r1) {
      t_next = p.t[row + 1];
      tp_next = p.tp[row + 1];
    }
    float A = 0.0f, P = 0.0f, R = 0.0f;
    {
      Inputs x;
      take(slot, x);
      add_sums(x, w, m, t, A, P, R);
    }
    row_totals(A, P, R, red, turn);
    asm volatile("" ::: "memory");   // (read again: the row's 64 values do not stay in registers meanwhile)
    {
      Inputs x;
      take(slot, x);
      finish<T>(p, row, c, n, x, w, m, factors(t, tp, A, P, R, mean), sw, sn, vec);
    }
    fetch(row + depth, slot);
    slot = slot + 1 == depth ? 0 : slot + 1;
    if (p.partial && (row + 1 == r1 || row + 1 == group_end)) {
      if (n > 0) flush<T>(p, group, r0, r1, c, n, sn, first, vec);
      first = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = both(0.0f);
    }
  }
  copies_wait(0);
  if (p.partial && n > 0) store_part(part(p, blockIdx.x, kDw, c), sw);
}

// Rows of more than 8192 elements, in segments of that many, read twice.  The sums over rows are kept in this CTA's rows
// of the workspace, that of H a tp in kTail until its gate row ends.
template <class T>
__global__ void __launch_bounds__(kRowThreads, 1) sandwich_backward_long_kernel(const SandwichGradParams p, const Split split,
                                                                                const uint32_t vec) {
  __shared__ float red[2][4][16];
  griddep_wait();
  griddep_launch_dependents();
  const unsigned r0 = blockIdx.x * split.rows;
  const unsigned r1 = static_cast<unsigned>(min(static_cast<int64_t>(r0) + split.rows, p.rows));
  const float mean = 1.0f / static_cast<float>(p.cols);
  int turn = 0;
  bool first = true;
  Inputs x;
  float2 w[8], m[8];
  const auto load = [&](unsigned row, unsigned group, int64_t c) {
    const int n = static_cast<int>(min(int64_t(16), p.cols - c));
    unpack(load16(static_cast<const T *>(p.dy) + row * p.lddy + c, n, level(vec, 0)), x.dy);
    if (p.dh) {
      unpack(load16(static_cast<const T *>(p.dh) + row * p.lddh + c, n, level(vec, 1)), x.dh);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.dh[i] = both(0.0f);
    }
    const auto matrix = [&](const Kept &k, int lv, float2 (&v)[8]) {
      if (k.s)
        unpack_kept(load16_fp8(static_cast<const unsigned char *>(k.p) + row * k.ld + c, n, lv), k.s[row * k.lds + (c >> 7)],
                    k.e5m2, v);
      else
        unpack(load16(static_cast<const T *>(k.p) + row * k.ld + c, n, lv), v);
    };
    matrix(p.a, level(vec, 7), x.a);
    matrix(p.h, level(vec, 8), x.h);
    load16_w<T>(p.w, p.w_f32, c, n, level(vec, 2), w);
    load_gated<T>(p, group, c, n, vec, m);
    return n;
  };
  for (unsigned row = r0; row < r1; ++row) {
    const float t = p.t[row], tp = p.tp[row];
    const unsigned group = p.gate.p ? row / p.gate.rows : 0;
    float A = 0.0f, P = 0.0f, R = 0.0f;
    for (int64_t c = threadIdx.x * 16; c < p.cols; c += kRowElements) {
      load(row, group, c);
      add_sums(x, w, m, t, A, P, R);
    }
    row_totals(A, P, R, red, turn);
    const Factors f = factors(t, tp, A, P, R, mean);
    const bool begins = row == r0 || (p.gate.p && row % p.gate.rows == 0);
    const bool ends = row + 1 == r1 || (p.gate.p && (row + 1) % p.gate.rows == 0);
    for (int64_t c = threadIdx.x * 16; c < p.cols; c += kRowElements) {
      const int n = load(row, group, c);
      float2 sw[8], sn[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sw[i] = sn[i] = both(0.0f);
      if (p.partial && row > r0) load_part(part(p, blockIdx.x, kDw, c), sw);
      if (p.partial && !begins) load_part(part(p, blockIdx.x, kTail, c), sn);
      finish<T>(p, row, c, n, x, w, m, f, sw, sn, vec);
      if (!p.partial) continue;
      store_part(part(p, blockIdx.x, kDw, c), sw);
      if (ends)
        flush<T>(p, group, r0, r1, c, n, sn, first, vec);
      else
        store_part(part(p, blockIdx.x, kTail, c), sn);
    }
    if (ends) first = false;
  }
}

// Sums over CTAs in a fixed order: blockIdx.y 0 of dw, 1 of dwp, then of the gate rows that several CTAs share, which
// are found by the gate row (by_group) or by the boundary between two CTAs.
template <class T>
__global__ void __launch_bounds__(1024) sandwich_sums_kernel(const SandwichGradParams p, const Split split,
                                                             const bool by_group) {
  __shared__ float red[32][33];
  griddep_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
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
  const auto kind = [&](unsigned b) {
    return blockIdx.y == 0   ? kDw
           : blockIdx.y == 1 ? kDwp
           : static_cast<int64_t>(group) * p.gate.rows < static_cast<int64_t>(b) * split.rows ? kHead
                                                                                              : kTail;
  };
  float sum = 0.0f;
  for (unsigned b0 = first + threadIdx.y; b0 < end; b0 += 160) {   // five loads in flight
    float v[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = c < p.cols && b0 + 32 * i < end ? *part(p, b0 + 32 * i, kind(b0 + 32 * i), c) : 0.0f;
#pragma unroll
    for (int i = 0; i < 5; ++i) sum += v[i];
  }
  red[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  sum = red[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
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

template <class T, bool KA, bool KH>
cudaError_t rows_kernel(const SandwichGradParams &p, const RowsShape &g, uint32_t vec, cudaStream_t s) {
  struct Tag {};
  const cudaError_t err = allow_smem<Tag>(sandwich_backward_kernel<T, KA, KH>);
  if (err != cudaSuccess) return err;
  const int row_bytes = RowPlaces<T, KA, KH>::kBytes * g.threads, depth = rows_ahead(g, row_bytes);
  return launch_maybe_pdl(sandwich_backward_kernel<T, KA, KH>, dim3(g.split.ctas), dim3(g.threads),
                          static_cast<size_t>(depth) * row_bytes, s, true, p, g.split, depth, vec);
}

template <class T>
cudaError_t typed(const SandwichGradParams &p, cudaStream_t s, int *launches) {
  const bool sums = p.dw || p.dwp || p.dgate;
  const RowsShape g = rows_shape(p.rows, p.cols, kSms);
  constexpr int e = sizeof(T);
  const int ew = p.w_f32 ? 4 : e, eg = p.gate.f32 ? 4 : e;
  const uint32_t vec = level_of(p.dy, p.lddy, e, 0) | level_of(p.dh, p.lddh, e, 1) | level_of(p.w, 0, ew, 2) |
                       level_of(p.wp, 0, ew, 3) | level_of(p.gate.p, p.gate.ld, eg, 4) | level_of(p.da, p.ldda, e, 5) |
                       level_of(p.dx, p.lddx, e, 6) | level_of(p.a.p, p.a.ld, p.a.s ? 1 : e, 7) |
                       level_of(p.h.p, p.h.ld, p.h.s ? 1 : e, 8) | level_of(p.dgate, p.lddgate, eg, 9);
  if (p.rows > 0) {
    cudaError_t err;
    if (g.segments)
      err = launch_maybe_pdl(sandwich_backward_long_kernel<T>, dim3(g.split.ctas), dim3(g.threads), 0, s, true, p, g.split, vec);
    else if (p.a.s)
      err = p.h.s ? rows_kernel<T, true, true>(p, g, vec, s) : rows_kernel<T, true, false>(p, g, vec, s);
    else
      err = p.h.s ? rows_kernel<T, false, true>(p, g, vec, s) : rows_kernel<T, false, false>(p, g, vec, s);
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

int64_t sandwich_partials(int64_t rows, int64_t cols) {
  return static_cast<int64_t>(rows_shape(rows, cols, kSms).split.ctas) * kParts * part_pitch(cols);
}

cudaError_t launch_sandwich_norm_backward(const SandwichGradParams &p, cudaStream_t s, int *launches) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return typed<float>(p, s, launches);
    case SGEMM_TYPE_BF16: return typed<__nv_bfloat16>(p, s, launches);
    default: return typed<__half>(p, s, launches);
  }
}

}  // namespace sg
