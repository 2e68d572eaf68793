// sandwich_forward.cuh -- the norms around a block, with a quantised output: one instance of the file for each type.
// 8192 x 8192 bf16 with checkpoints 138 us, 4.4 TB/s, without 88 us, 5.4 TB/s: 42 instructions an element at 54 % of the issue
// slots (some of them spills, see the kernel), and the two sums' latencies.
#pragma once

#include <type_traits>

#include "sandwich_norm.cuh"

namespace sg {
namespace {

// What a row's outputs need of 16 of its elements.
struct Outputs {
  float2 na[8], h[8], y[8];   // -a, h, y
};

// Stores h, y quantised and, with KEEP, the checkpoints of a and h, and their blocks' scales.  KEEP: 0 none, 1 E4M3,
// 2 E5M2.  c: the first element's column.  vec: 5 h, 6 q, 7 qa, 8 qh.
template <class T, bool E5M2, int KEEP, class C>
__device__ __forceinline__ void store_outputs(const SandwichParams &p, int64_t row, C c, int n, Outputs &o, uint32_t vec) {
  const int lane8 = threadIdx.x & 7;
  const C block = c >> 7;
  const bool live = static_cast<int64_t>(block) * 128 < p.cols;
  if (n < 16) {   // a row with a NaN or an infinity must not reach past its end
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (2 * i >= n) o.h[i].x = o.y[i].x = 0.0f;
      if (2 * i + 1 >= n) o.h[i].y = o.y[i].y = 0.0f;
    }
  }
  store16(static_cast<T *>(p.h) + row * p.ldh + c, o.h, n, level(vec, 5));
  float scale;
  int own = 0;
  if (KEEP) {
    const float m[4] = {max_abs16(o.y), max_abs16(o.h), max_abs16(o.na), 0.0f};
    own = owned_by(lane8);
    scale = scale_of(owned_max(m, lane8), own == 0 ? E5M2 : KEEP == 2);
  } else {
    scale = scale_of(max_of_8(max_abs16(o.y)), E5M2);
  }
  const auto of = [&](float v, int i) { return KEEP ? __shfl_sync(~0u, v, owner_of(i), 8) : v; };
  const float inv = inv_of(scale);
  store16_fp8(p.q + row * p.ldq + c, quantise<E5M2>(o.y, of(inv, 0)), n, level(vec, 6));
  if (lane8 == owner_of(0) && live) p.s[row * p.lds + block] = scale;
  if (KEEP) {
    const float div = divisor(scale), ninv = ninv_of(scale);
    const float dh = of(div, 1), nh = of(ninv, 1), da = of(div, 2), na = of(ninv, 2);
    if (p.qh) {   // (as the quantiser does, bit for bit: 8192 x 8192 136.6 us, by the product with 1 / s rounded 135.6)
#pragma unroll
      for (int i = 0; i < 8; ++i) o.h[i] = mul2(o.h[i], both(-1.0f));
      store16_fp8(p.qh + row * p.ldqh + c, quantise_exactly<KEEP == 2>(o.h, dh, nh), n, level(vec, 8));
      if (lane8 == owner_of(1) && live) p.sh[row * p.ldsh + block] = scale;
    }
    if (p.qa) {
      store16_fp8(p.qa + row * p.ldqa + c, quantise_exactly<KEEP == 2>(o.na, da, na), n, level(vec, 7));
      if (lane8 == owner_of(2) && live) p.sa[row * p.ldsa + block] = scale;
    }
  }
}

// gate wp (a gate's row) of sixteen columns.
template <class T>
__device__ __forceinline__ void load_gated(const void *wp, bool w_f32, const Gate &gate, int64_t gate_row, int64_t c, int n,
                                           int lw, int lg, float2 (&m)[8]) {
  load16_w<T>(wp, w_f32, c, n, lw, m);
  if (gate.p) {
    float2 g[8];
    load16_w<T>(gate.p, gate.f32, gate_row * gate.ld + c, n, lg, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = mul2(m[i], g[i]);
  }
}

__device__ __forceinline__ float square_sum(const float2 (&v)[8]) {
  float2 s = mul2(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) s = fma2(v[i], v[i], s);
  return s.x + s.y;
}

// A thread holds N times 16 consecutive elements of a row (or of a segment of it): one, with 64 registers, or two, with 80,
// which divides a thread's fixed work (sums, offsets) by more elements and lets three rows of 8192 share an SM, but leaves
// few rows less parallel.  Up to 5120 columns three rows or more share an SM either way.  One against two, in us, when they
// were compared: 8192 x 8192 bf16 with checkpoints 144 and 135, without 103 and 88; 4072 x 6144 F16 62.5 and 54.8, 52.7 and
// 42.2; 4072 x 5120 47.6 and 50.6, 39.4 and 39.1; 4072 x 4224 44.9 and 49.5, 37.3 and 38.2; 512 x 4096 5.6 and 7.8; 4096 x 8192
// F32 118 and 138.
// These registers do not hold everything.  Bytes that a thread spills and loads again: two chunks with checkpoints 72 and 108
// (bf16), 104 and 208 (F16), one chunk at most 60 and 60, but 224 and 144 of F32 with checkpoints and 400 and 128 of its longer
// rows; without checkpoints otherwise at most 48 and 48.
// FORM: kWarps, a row a warp and eight rows a CTA; kOne, a row a CTA; kLong, rows of more than 16384 elements, in segments
// of that many: a three times, x twice from memory (or the L2 cache).  (A row that is the same for the whole CTA is left to
// the uniform data path, with its offsets.)  vec: 0 a, 1 x, 2 w, 3 wp, 4 gate, and see store_outputs
enum : int { kWarps = 0, kOne = 1, kLong = 2 };
template <class T, bool E5M2, int KEEP, int FORM, int N>
__global__ void __launch_bounds__(N == 1 ? kRowThreads : kPairThreads, N == 1 ? 1 : 3)
    sandwich_norm_kernel(const SandwichParams p, const uint32_t vec) {
  using Col = std::conditional_t<FORM == kLong, int64_t, int>;
  __shared__ __align__(16) float red[2][1][32];
  griddep_wait();
  griddep_launch_dependents();
  RowSums<1> row_sums(red);
  const int64_t row = FORM == kWarps ? static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y : blockIdx.x;
  if (FORM == kWarps && row >= p.rows) return;   // (whole warps)
  const unsigned group = p.gate.p ? static_cast<unsigned>(row) / p.gate.rows : 0;
  const T *a = static_cast<const T *>(p.a) + row * p.lda, *x = static_cast<const T *>(p.x) + row * p.ldx;
  const float mean = 1.0f / static_cast<float>(p.cols);
  const Col cols = static_cast<Col>(p.cols), end = FORM == kLong ? cols : 1;
  const auto column = [&](Col base, int j) { return base + (static_cast<Col>(threadIdx.x) + j * static_cast<Col>(blockDim.x)) * 16; };
  const auto count = [&](Col base, int j) { return static_cast<int>(max(Col(0), min(Col(16), cols - column(base, j)))); };
  Raw16<T> ra[N], rx[N];
  const auto load = [&](Col base, bool with_x) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const Col c = column(base, j);
      ra[j] = load16(a + c, count(base, j), level(vec, 0), inside(c, cols));
      if (with_x) rx[j] = load16(x + c, count(base, j), level(vec, 1), inside(c, cols));
    }
  };
  load(0, true);
  float sum[1] = {0.0f};
  for (Col base = 0; base < end; base += kRowElements) {
    if (FORM == kLong) load(base, false);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float2 v[8];
      ra[j] = negated(ra[j]);   // (the exact quotients of its checkpoint want -a)
      unpack(ra[j], v);
      sum[0] += square_sum(v);
    }
  }
  row_sums(sum);
  const float tp = rsqrtf(fmaf(sum[0], mean, p.eps));
  float2 h[N][8];
  const auto make_h = [&](Col base) {
    if (FORM == kLong) load(base, true);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float2 m[8], v[8];
      load_gated<T>(p.wp, p.w_f32, p.gate, group, column(base, j), count(base, j), level(vec, 3), level(vec, 4), m);
      if (FORM == kLong) ra[j] = negated(ra[j]);
      unpack(ra[j], v);
      unpack(rx[j], h[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = fma2(both(p.residual_scale), h[j][i], mul2(mul2(v[i], both(-tp)), m[i]));
    }
  };
  sum[0] = 0.0f;
  for (Col base = 0; base < end; base += kRowElements) {
    make_h(base);
#pragma unroll
    for (int j = 0; j < N; ++j) sum[0] += square_sum(h[j]);
  }
  row_sums(sum);
  const float t = rsqrtf(fmaf(sum[0], mean, p.eps));
  if (threadIdx.x == 0) {
    if (p.tp) p.tp[row] = tp;
    if (p.t) p.t[row] = t;
  }
  for (Col base = 0; base < end; base += kRowElements) {   // (whole warps: the blocks' lanes stay together)
    if (FORM == kLong) make_h(base);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Outputs o;
      float2 w[8];
      load16_w<T>(p.w, p.w_f32, column(base, j), count(base, j), level(vec, 2), w);
      unpack(ra[j], o.na);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o.h[i] = h[j][i];
        o.y[i] = mul2(mul2(h[j][i], both(t)), w[i]);
      }
      store_outputs<T, E5M2, KEEP>(p, row, column(base, j), count(base, j), o, vec);
    }
  }
}

template <class T, bool E5M2, int KEEP>
cudaError_t launch(const SandwichParams &p, int sm_count, cudaStream_t s) {
  constexpr int e = sizeof(T);
  const int ew = p.w_f32 ? 4 : e, eg = p.gate.f32 ? 4 : e;
  const uint32_t vec = level_of(p.a, p.lda, e, 0) | level_of(p.x, p.ldx, e, 1) | level_of(p.w, 0, ew, 2) |
                       level_of(p.wp, 0, ew, 3) | level_of(p.gate.p, p.gate.ld, eg, 4) | level_of(p.h, p.ldh, e, 5) |
                       level_of(p.q, p.ldq, 1, 6) | level_of(p.qa, p.ldqa, 1, 7) | level_of(p.qh, p.ldqh, 1, 8);
  const int64_t chunks = (p.cols + 15) / 16;
  if constexpr (e == 2) {
    if (p.cols > 5120 && p.cols <= 32 * kPairThreads && p.rows >= 8 * sm_count)
      return launch_maybe_pdl(sandwich_norm_kernel<T, E5M2, KEEP, kOne, 2>, dim3(static_cast<unsigned>(p.rows)),
                              dim3(static_cast<unsigned>((chunks + 63) / 64 * 32)), 0, s, true, p, vec);
  }
  const int threads = row_threads(p.cols), rows = threads == 32 ? 8 : 1;   // of a CTA
  const dim3 grid(static_cast<unsigned>((p.rows + rows - 1) / rows)), block(threads, rows);
  const auto kernel = threads == 32             ? sandwich_norm_kernel<T, E5M2, KEEP, kWarps, 1>
                      : p.cols <= kRowElements ? sandwich_norm_kernel<T, E5M2, KEEP, kOne, 1>
                                               : sandwich_norm_kernel<T, E5M2, KEEP, kLong, 1>;
  return launch_maybe_pdl(kernel, grid, block, 0, s, true, p, vec);
}

}  // namespace

template <class T>
cudaError_t launch_norms(const SandwichParams &p, int sm_count, cudaStream_t s) {
  if (!(p.qa || p.qh)) return p.e5m2 ? launch<T, true, 0>(p, sm_count, s) : launch<T, false, 0>(p, sm_count, s);
  if (p.keep_e5m2) return p.e5m2 ? launch<T, true, 2>(p, sm_count, s) : launch<T, false, 2>(p, sm_count, s);
  return p.e5m2 ? launch<T, true, 1>(p, sm_count, s) : launch<T, false, 1>(p, sm_count, s);
}

}  // namespace sg
