// sandwich_norm.cu -- the norms around a block, with a quantised output.
#include "sandwich_norm.cuh"

namespace sg {
namespace {

// What a row's outputs need of 16 of its elements: a, h and the norm's factor of them.
struct Outputs {
  float2 a[8], h[8], y[8];
};

// Stores h, y quantised and, with KEEP, the checkpoints of a and h, and their blocks' scales.  KEEP: 0 none, 1 E4M3,
// 2 E5M2.  c: the first element's column.  vec: 5 h, 6 q, 7 qa, 8 qh.
template <class T, bool E5M2, int KEEP>
__device__ __forceinline__ void store_outputs(const SandwichParams &p, int64_t row, int64_t c, int n, Outputs &o, uint32_t vec) {
  const int lane8 = threadIdx.x & 7;
  const int64_t block = c >> 7;
  const bool live = block * 128 < p.cols;
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
    const float m[4] = {max_abs16(o.y), max_abs16(o.h), max_abs16(o.a), 0.0f};
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
    const float ih = of(inv, 1), da = of(divisor(scale), 2), na = of(ninv_of(scale), 2);
    if (p.qh) {
      store16_fp8(p.qh + row * p.ldqh + c, quantise<KEEP == 2>(o.h, ih), n, level(vec, 8));
      if (lane8 == owner_of(1) && live) p.sh[row * p.ldsh + block] = scale;
    }
    if (p.qa) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o.a[i] = make_float2(-o.a[i].x, -o.a[i].y);
      store16_fp8(p.qa + row * p.ldqa + c, quantise_exactly<KEEP == 2>(o.a, da, na), n, level(vec, 7));
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

// vec: 0 a, 1 x, 2 w, 3 wp, 4 gate, and see store_outputs
template <class T, bool E5M2, int KEEP>
__global__ void __launch_bounds__(kRowThreads, 1) sandwich_norm_kernel(const SandwichParams p, const Split split,
                                                                       const int depth, const uint32_t vec) {
  constexpr int U = sizeof(T);
  extern __shared__ __align__(16) uint4 rows_smem[];   // [depth][a, x][U][thread]
  __shared__ float red[2][16];
  griddep_wait();
  griddep_launch_dependents();
  const int step = blockDim.x;
  const unsigned r0 = blockIdx.x * split.rows;
  const unsigned r1 = static_cast<unsigned>(min(static_cast<int64_t>(r0) + split.rows, p.rows));
  const int64_t c = threadIdx.x * 16;
  const int n = static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - c)));
  uint4 *mine = rows_smem + threadIdx.x;
  const auto fetch = [&](unsigned row, int slot) {
    if (row < r1) {
      uint4 *to = mine + slot * 2 * U * step;
      copy16(to, step, static_cast<const T *>(p.a) + row * p.lda + c, n, level(vec, 0));
      copy16(to + U * step, step, static_cast<const T *>(p.x) + row * p.ldx + c, n, level(vec, 1));
    }
    copies_commit();
  };
  for (int d = 0; d < depth; ++d) fetch(r0 + d, d);
  float2 w[8], m[8];
  load16_w<T>(p.w, p.w_f32, c, n, level(vec, 2), w);
  unsigned group = p.gate.p ? r0 / p.gate.rows : 0, group_end = p.gate.p ? (group + 1) * p.gate.rows : ~0u;
  load_gated<T>(p.wp, p.w_f32, p.gate, group, c, n, level(vec, 3), level(vec, 4), m);
  const float mean = 1.0f / static_cast<float>(p.cols);
  int turn = 0, slot = 0;
  for (unsigned row = r0; row < r1; ++row) {
    if (row >= group_end) {
      ++group;
      group_end += p.gate.rows;
      load_gated<T>(p.wp, p.w_f32, p.gate, group, c, n, level(vec, 3), level(vec, 4), m);
    }
    copies_wait(depth - 1);
    Outputs o;
    const uint4 *at = mine + slot * 2 * U * step;
    unpack(take16<T>(at, step), o.a);
    const Raw16<T> x = take16<T>(at + U * step, step);
    fetch(row + depth, slot);
    slot = slot + 1 == depth ? 0 : slot + 1;
    const float tp = 1.0f / sqrtf(fmaf(row_total(square_sum(o.a), red, turn), mean, p.eps));
    unpack(x, o.h);
#pragma unroll
    for (int i = 0; i < 8; ++i) o.h[i] = fma2(both(p.residual_scale), o.h[i], mul2(mul2(o.a[i], both(tp)), m[i]));
    const float t = 1.0f / sqrtf(fmaf(row_total(square_sum(o.h), red, turn), mean, p.eps));
    if (threadIdx.x == 0) {
      if (p.tp) p.tp[row] = tp;
      if (p.t) p.t[row] = t;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) o.y[i] = mul2(mul2(o.h[i], both(t)), w[i]);
    store_outputs<T, E5M2, KEEP>(p, row, c, n, o, vec);
  }
  copies_wait(0);
}

// Rows of more than 8192 elements, in segments of that many: a three times, x twice from memory (or the L2 cache).
template <class T, bool E5M2, int KEEP>
__global__ void __launch_bounds__(kRowThreads, 1) sandwich_norm_long_kernel(const SandwichParams p, const uint32_t vec) {
  __shared__ float red[2][16];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const unsigned group = p.gate.p ? static_cast<unsigned>(row) / p.gate.rows : 0;
  const T *a = static_cast<const T *>(p.a) + row * p.lda, *x = static_cast<const T *>(p.x) + row * p.ldx;
  const float mean = 1.0f / static_cast<float>(p.cols);
  int turn = 0;
  const auto count = [&](int64_t c) { return static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - c))); };
  float sum = 0.0f;
  for (int64_t c = threadIdx.x * 16; c < p.cols; c += kRowElements) {
    float2 v[8];
    unpack(load16(a + c, count(c), level(vec, 0)), v);
    sum += square_sum(v);
  }
  const float tp = 1.0f / sqrtf(fmaf(row_total(sum, red, turn), mean, p.eps));
  const auto make_h = [&](int64_t c, Outputs &o) {
    const int n = count(c);
    float2 m[8];
    unpack(load16(a + c, n, level(vec, 0)), o.a);
    unpack(load16(x + c, n, level(vec, 1)), o.h);
    load_gated<T>(p.wp, p.w_f32, p.gate, group, c, n, level(vec, 3), level(vec, 4), m);
#pragma unroll
    for (int i = 0; i < 8; ++i) o.h[i] = fma2(both(p.residual_scale), o.h[i], mul2(mul2(o.a[i], both(tp)), m[i]));
  };
  Outputs o;
  sum = 0.0f;
  for (int64_t c = threadIdx.x * 16; c < p.cols; c += kRowElements) {
    make_h(c, o);
    sum += square_sum(o.h);
  }
  const float t = 1.0f / sqrtf(fmaf(row_total(sum, red, turn), mean, p.eps));
  if (threadIdx.x == 0) {
    if (p.tp) p.tp[row] = tp;
    if (p.t) p.t[row] = t;
  }
  for (int64_t base = 0; base < p.cols; base += kRowElements) {   // (whole warps: the blocks' lanes stay together)
    const int64_t c = base + threadIdx.x * 16;
    float2 w[8];
    make_h(c, o);
    load16_w<T>(p.w, p.w_f32, c, count(c), level(vec, 2), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) o.y[i] = mul2(mul2(o.h[i], both(t)), w[i]);
    store_outputs<T, E5M2, KEEP>(p, row, c, count(c), o, vec);
  }
}

template <class T, bool E5M2, int KEEP>
cudaError_t launch(const SandwichParams &p, int sm_count, cudaStream_t s) {
  constexpr int e = sizeof(T);
  const int ew = p.w_f32 ? 4 : e, eg = p.gate.f32 ? 4 : e;
  const uint32_t vec = level_of(p.a, p.lda, e, 0) | level_of(p.x, p.ldx, e, 1) | level_of(p.w, 0, ew, 2) |
                       level_of(p.wp, 0, ew, 3) | level_of(p.gate.p, p.gate.ld, eg, 4) | level_of(p.h, p.ldh, e, 5) |
                       level_of(p.q, p.ldq, 1, 6) | level_of(p.qa, p.ldqa, 1, 7) | level_of(p.qh, p.ldqh, 1, 8);
  const RowsShape g = rows_shape(p.rows, p.cols, sm_count);
  if (g.segments)
    return launch_maybe_pdl(sandwich_norm_long_kernel<T, E5M2, KEEP>, dim3(static_cast<unsigned>(p.rows)), dim3(kRowThreads),
                            0, s, true, p, vec);
  struct Tag {};
  const cudaError_t err = allow_smem<Tag>(sandwich_norm_kernel<T, E5M2, KEEP>);
  if (err != cudaSuccess) return err;
  const int row_bytes = 2 * e * 16 * g.threads, depth = rows_ahead(g, row_bytes);
  return launch_maybe_pdl(sandwich_norm_kernel<T, E5M2, KEEP>, dim3(g.split.ctas), dim3(g.threads),
                          static_cast<size_t>(depth) * row_bytes, s, true, p, g.split, depth, vec);
}

template <class T>
cudaError_t typed(const SandwichParams &p, int sm_count, cudaStream_t s) {
  if (!(p.qa || p.qh)) return p.e5m2 ? launch<T, true, 0>(p, sm_count, s) : launch<T, false, 0>(p, sm_count, s);
  if (p.keep_e5m2) return p.e5m2 ? launch<T, true, 2>(p, sm_count, s) : launch<T, false, 2>(p, sm_count, s);
  return p.e5m2 ? launch<T, true, 1>(p, sm_count, s) : launch<T, false, 1>(p, sm_count, s);
}

}  // namespace

cudaError_t launch_sandwich_norm(const SandwichParams &p, int sm_count, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return typed<float>(p, sm_count, s);
    case SGEMM_TYPE_BF16: return typed<__nv_bfloat16>(p, sm_count, s);
    default: return typed<__half>(p, sm_count, s);
  }
}

}  // namespace sg
