// sandwich_backward.cu -- the gradient of the norms around a block
// (sandwich_norm.cuh has the formulas).
//
// A row is 16 consecutive elements a thread, 128 threads a CTA and, where it
// has more than 2048 elements, up to eight CTAs of a cluster.  A cluster takes
// consecutive rows one after the other: a row's values and the sums over rows
// stay in registers (96 of a thread's 128), the weights in places of the
// thread's own in shared memory, where it also copies its elements of the next
// row as soon as it has taken this one's.  An SM's four CTAs belong to different
// rows, which are in different phases.  (With the weights in registers and every
// row read and unpacked twice, 4095 x 8192 from checkpoints took 101 us, so 86, 3.9 TB/s;
// two rows copied ahead 89.)
//
// The second mean is that of a sum which is linear in the first, so both come
// from three sums over the row, taken together:
//   A = sum dy w h,  P = sum (t dy w + dh) p,  R = sum h p   with p = gate wp a
//   sum v a = P - t^3 (A / cols) R
#include <mutex>

#include "sandwich_norm.cuh"

namespace sg {
namespace {

constexpr int kSms = 152;   // of a GB300: sizes the partial sums, whose number must not depend on the device
constexpr int kClusterThreads = 128, kMaxCluster = 8;   // of a CTA; CTAs of a row
constexpr int kLongThreads = 512, kLongElements = 16 * kLongThreads;   // of a segment of a longer row

// Clusters, each with `rows` consecutive rows (the last one fewer), and their CTAs.
struct Split {
  unsigned clusters, rows, cluster;
};

// The workspace: for every cluster a row of `pitch` floats for each of dw, dwp, and dgate's sums over the rows of the first
// and of the last gate row that it shares with other clusters.
enum : int { kDw = 0, kDwp = 1, kHead = 2, kTail = 3, kParts = 4 };
inline __host__ __device__ int64_t part_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }
__device__ __forceinline__ float *part(const SandwichGradParams &p, unsigned stream, int kind, int64_t c) {
  return p.partial + (static_cast<int64_t>(stream) * kParts + kind) * part_pitch(p.cols) + c;
}
__device__ __forceinline__ void load_part(const float *at, float2 (&v)[8]) { unpack(load16(at, 16, 1), v); }
__device__ __forceinline__ void store_part(float *at, const float2 (&v)[8]) { store16(at, v, 16, 1); }

// The three sums of a row over its threads, in a fixed order: in a warp as in RowSums, then every warp leaves its sums with
// every CTA of the cluster, by stores that count towards an mbarrier there (a cluster barrier would wait for the stores to
// memory, too: 8192 x 8192 284 instead of 254 us).  Used by turns, so that nothing is overwritten that a slower warp still
// reads: a warp's sums of call i + 1 show that it has read those of call i.
struct ClusterTotals {
  float red[2][4][32];   // [turn][value][warp]; zero where there is none
  uint64_t bar[2];
};
class ClusterSums {
  ClusterTotals *sh;
  unsigned cluster, calls = 0;
  bool ok = true;
  uint64_t budget_ns;
  int *status;

 public:
  unsigned rank;

  __device__ __forceinline__ ClusterSums(ClusterTotals *shared, unsigned cluster_size, uint64_t budget, int *device_status)
      : sh(shared), cluster(cluster_size), budget_ns(budget), status(device_status),
        rank(cluster_size > 1 ? cluster_ctarank() : 0) {
    for (int i = threadIdx.x; i < 2 * 4 * 32; i += blockDim.x) (&sh->red[0][0][0])[i] = 0.0f;
    if (cluster > 1) {
      if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sh->bar[0]), 1);
        mbar_init(smem_u32(&sh->bar[1]), 1);
        fence_mbar_init();
      }
      cluster_sync();   // (every CTA of the cluster is there to be written to)
    } else {
      __syncthreads();
    }
  }
  // False (for the whole warp) if the other warps' sums did not come in time.  The warp then sends and expects nothing more
  // and the caller leaves its loop, so that the others run out of time as well and come to finish().
  __device__ __forceinline__ bool operator()(float (&v)[4]) {
    const int lane = threadIdx.x & 31, own = lane / 8, j = lane % 8;
#pragma unroll
    for (int k = 2, d = 16; k > 0; k >>= 1, d >>= 1) {
      const bool upper = lane & d;
#pragma unroll
      for (int i = 0; i < k; ++i) {
        const float mine = upper ? v[k + i] : v[i], give = upper ? v[i] : v[k + i];
        v[i] = mine + __shfl_xor_sync(~0u, give, d);
      }
    }
    float s = v[0];
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    const unsigned warps = blockDim.x >> 5, turn = calls & 1;
    if (cluster > 1 || warps > 1) {
      float *to = &sh->red[turn][own][rank * warps + (threadIdx.x >> 5)];
      if (cluster > 1) {
        const uint32_t bar = smem_u32(&sh->bar[turn]);
        if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, cluster * warps * 16);
        if (j < static_cast<int>(cluster))
          asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                           map_to_rank(smem_u32(to), j)),
                       "r"(__float_as_uint(s)), "r"(map_to_rank(bar, j))
                       : "memory");
        ok = __all_sync(~0u, wait_parity_bounded(bar, calls >> 1 & 1, budget_ns, status, SharedOfCluster()));
        if (!ok) return false;
      } else {
        if (j == 0) *to = s;
        __syncthreads();
      }
      const float4 u = *reinterpret_cast<const float4 *>(&sh->red[turn][own][4 * j]);
      s = (u.x + u.y) + (u.z + u.w);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      ++calls;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(~0u, s, 8 * i);
    return true;
  }
  // Before the CTA ends: no warp of the cluster sends anything more, and what was sent has arrived (it was waited for; after
  // a wait that ran out, some time is given to it).
  __device__ __forceinline__ void finish() {
    if (cluster == 1) return;
    cluster_sync();
    if (!ok)
      for (int i = 0; i < 100; ++i) __nanosleep(1000);
  }
};

// Whether all rows have one gate (or none): then dwp and dgate follow from one sum, which lies in dwp's place.
__host__ __device__ inline bool one_gate(const SandwichGradParams &p) { return !p.gate.p || p.gate.rows >= p.rows; }

// What a row's sums over rows add up to at the end of a cluster's (`stream`'s) rows r0 .. r1 - 1 of a gate row (`group`): its
// part of dwp is added to the cluster's, and its part of dgate is stored, or dgate itself if all its rows are here.
template <class T>
__device__ __forceinline__ void flush(const SandwichGradParams &p, unsigned stream, unsigned group, unsigned r0, unsigned r1, int64_t c, int n,
                                      const float2 (&sn)[8], bool first, uint32_t vec) {
  if (one_gate(p)) {
    store_part(part(p, stream, kDwp, c), sn);
    return;
  }
  float2 v[8];
  load16_w<T>(p.gate.p, p.gate.f32, group * p.gate.ld + c, n, level(vec, 4), v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], sn[i]);
  float *dwp = part(p, stream, kDwp, c);
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
    store_part(part(p, stream, g0 < r0 ? kHead : kTail, c), sn);
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
// KIND: 1 E4M3, 2 E5M2, 3 one of them
template <int KIND>
__device__ __forceinline__ void unpack_kept(uint4 u, float scale, bool e5m2, float2 (&v)[8]) {
  if (KIND == 3 ? e5m2 : KIND == 2)
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
// An infinite scale of a checkpoint makes NaN of the zeros behind a row's end, which are not of the row's sums.
__device__ __forceinline__ void clear_kept(Inputs &x, int n) {
  if (n >= 16) return;
  clear_from(x.a, n);
  clear_from(x.h, n);
}
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

// Sixteen floats of this thread's own in shared memory.
__device__ __forceinline__ void load_own(const float4 *at, float2 (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 u = at[k * kUnitStep];
    v[2 * k] = make_float2(u.x, u.y);
    v[2 * k + 1] = make_float2(u.z, u.w);
  }
}
__device__ __forceinline__ void store_own(float4 *at, const float2 (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) at[k * kUnitStep] = make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
}

// KIND: a and h are 0 matrices of T, 1 checkpoints in E4M3, 2 in E5M2, 3 any of these, each its own.
// vec: 0 dy, 1 dh, 2 w, 3 wp, 4 gate, 5 da, 6 dx, 7 a, 8 h, 9 dgate
template <class T, int KIND>
struct RowPlaces {   // 16-byte units of a thread: w, gate wp, and the next row's inputs
  static constexpr int U = sizeof(T), K = KIND == 1 || KIND == 2 ? 1 : U;
  static constexpr int kGated = 4, kDy = 8, kDh = kDy + U, kA = kDh + U, kH = kA + K, kUnits = kH + K;
  static constexpr int kBytes = kUnits * 16 + 8;   // of a thread, with the scales of a and h
};
template <class T, int KIND>
__global__ void __launch_bounds__(kClusterThreads, 4) sandwich_backward_kernel(const SandwichGradParams p, const Split split,
                                                                           const uint32_t vec) {
  using At = RowPlaces<T, KIND>;
  extern __shared__ __align__(16) uint4 own_smem[];   // [warp][unit][lane], then [a's, h's scale][thread]
  __shared__ __align__(16) ClusterTotals shared;
  ClusterSums row_sums(&shared, split.cluster, p.wait_budget_ns, p.status);
  griddep_wait();
  griddep_launch_dependents();
  const unsigned stream = blockIdx.x / split.cluster;
  const unsigned r0 = stream * split.rows;
  const unsigned r1 = static_cast<unsigned>(min(static_cast<int64_t>(r0) + split.rows, p.rows));
  const unsigned c = (row_sums.rank * blockDim.x + threadIdx.x) * 16;
  const int n = max(0, min(16, static_cast<int>(p.cols) - static_cast<int>(c)));
  uint4 *mine = own_smem + first_unit(At::kUnits);
  float4 *weights = reinterpret_cast<float4 *>(mine), *gated = weights + At::kGated * kUnitStep;
  float *scales = reinterpret_cast<float *>(own_smem + blockDim.x * At::kUnits) + threadIdx.x;
  const bool in = inside(static_cast<int>(c), static_cast<int>(p.cols));
  // Whether the elements of every input are copied asynchronously.
  const bool fast = level(vec, 0) && (!p.dh || level(vec, 1)) &&
                    (KIND == 0 ? level(vec, 7) && level(vec, 8) : KIND < 3 && level(vec, 7) == 2 && level(vec, 8) == 2);
  if (n <= 0) {   // nothing is ever copied to these places
    for (int i = At::kDy; i < At::kUnits; ++i) mine[i * kUnitStep] = make_uint4(0, 0, 0, 0);
    scales[0] = scales[blockDim.x] = 0.0f;
  }
  const auto fetch = [&](unsigned row) {
    if (row < r1 && n > 0) {
      const T *dy = static_cast<const T *>(p.dy) + row * p.lddy + c, *dh = static_cast<const T *>(p.dh) + row * p.lddh + c;
      const auto aligned = [&](int n) {
        const auto matrix = [&](const Kept &k, uint4 *place, float *scale) {
          if (KIND == 0)
            copy16(place, static_cast<const T *>(k.p) + row * k.ld + c, n, 1);
          else
            copy16_kept(place, scale, static_cast<const unsigned char *>(k.p) + row * k.ld + c, k.s + row * k.lds + (c >> 7), n, 2);
        };
        copy16(mine + At::kDy * kUnitStep, dy, n, 1);
        if (p.dh) copy16(mine + At::kDh * kUnitStep, dh, n, 1);
        matrix(p.a, mine + At::kA * kUnitStep, scales);
        matrix(p.h, mine + At::kH * kUnitStep, scales + blockDim.x);
      };
      if (fast && n == 16) {
        aligned(16);
      } else if (fast) {
        aligned(n);
      } else {
        const auto matrix = [&](const Kept &k, int lv, uint4 *place, float *scale) {
          if (KIND == 3 ? k.s != nullptr : KIND != 0)
            copy16_kept(place, scale, static_cast<const unsigned char *>(k.p) + row * k.ld + c, k.s + row * k.lds + (c >> 7), n, lv);
          else
            copy16(place, static_cast<const T *>(k.p) + row * k.ld + c, n, lv, in);
        };
        copy16(mine + At::kDy * kUnitStep, dy, n, level(vec, 0), in);
        if (p.dh) copy16(mine + At::kDh * kUnitStep, dh, n, level(vec, 1), in);
        matrix(p.a, level(vec, 7), mine + At::kA * kUnitStep, scales);
        matrix(p.h, level(vec, 8), mine + At::kH * kUnitStep, scales + blockDim.x);
      }
    }
    copies_commit();
  };
  const auto take = [&](Inputs &x) {
    unpack(take16<T>(mine + At::kDy * kUnitStep), x.dy);
    if (p.dh) {
      unpack(take16<T>(mine + At::kDh * kUnitStep), x.dh);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.dh[i] = both(0.0f);
    }
    const auto matrix = [&](const Kept &k, const uint4 *place, const float *scale, float2 (&v)[8]) {
      if (KIND == 3 ? k.s != nullptr : KIND != 0)
        unpack_kept<KIND>(*place, *scale, k.e5m2, v);
      else
        unpack(take16<T>(place), v);
    };
    matrix(p.a, mine + At::kA * kUnitStep, scales, x.a);
    matrix(p.h, mine + At::kH * kUnitStep, scales + blockDim.x, x.h);
    if (KIND != 0) clear_kept(x, n);
  };
  fetch(r0);
  unsigned group = p.gate.p ? r0 / p.gate.rows : 0, group_end = p.gate.p ? (group + 1) * p.gate.rows : ~0u;
  const auto load_weights = [&] {
    float2 v[8];
    load_gated<T>(p, group, c, n, vec, v);
    store_own(gated, v);
  };
  load_weights();
  float2 sw[8], sn[8];
  load16_w<T>(p.w, p.w_f32, c, n, level(vec, 2), sw);
  store_own(weights, sw);
#pragma unroll
  for (int i = 0; i < 8; ++i) sw[i] = sn[i] = both(0.0f);
  const float mean = 1.0f / static_cast<float>(p.cols);
  bool first = true;
  float t_next = p.t[r0], tp_next = p.tp[r0];
  for (unsigned row = r0; row < r1; ++row) {
    if (row >= group_end) {
      ++group;
      group_end += p.gate.rows;
      load_weights();
    }
    copies_wait(0);
    Inputs x;
    take(x);
    fetch(row + 1);
    const float t = t_next, tp = tp_next;
    if (row + 1 < r1) {
      t_next = p.t[row + 1];
      tp_next = p.tp[row + 1];
    }
    float total[4] = {};
    {
      float2 w[8], m[8];
      load_own(weights, w);
      load_own(gated, m);
      add_sums(x, w, m, t, total[0], total[1], total[2]);
    }
    if (!row_sums(total)) break;
    asm volatile("" ::: "memory");   // (the weights are read again, they do not stay in registers meanwhile)
    {
      float2 w[8], m[8];
      load_own(weights, w);
      load_own(gated, m);
      finish<T>(p, row, c, n, x, w, m, factors(t, tp, total[0], total[1], total[2], mean), sw, sn, vec);
    }
    if (p.partial && (row + 1 == r1 || row + 1 == group_end)) {
      if (n > 0) flush<T>(p, stream, group, r0, r1, c, n, sn, first, vec);
      first = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = both(0.0f);
    }
  }
  copies_wait(0);
  if (p.partial && n > 0) store_part(part(p, stream, kDw, c), sw);
  row_sums.finish();
}

// Rows of more than 16384 elements, in segments of 8192, read twice.  The sums over rows are kept in this CTA's rows
// of the workspace, that of H a tp in kTail until its gate row ends.
template <class T>
__global__ void __launch_bounds__(kLongThreads, 1) sandwich_backward_long_kernel(const SandwichGradParams p, const Split split,
                                                                                const uint32_t vec) {
  __shared__ __align__(16) float red[2][4][32];
  griddep_wait();
  griddep_launch_dependents();
  RowSums<4> row_sums(red);
  const unsigned r0 = blockIdx.x * split.rows;
  const unsigned r1 = static_cast<unsigned>(min(static_cast<int64_t>(r0) + split.rows, p.rows));
  const float mean = 1.0f / static_cast<float>(p.cols);
  bool first = true;
  Inputs x;
  float2 w[8], m[8];
  const auto load = [&](unsigned row, unsigned group, int64_t c) {
    const int n = static_cast<int>(min(int64_t(16), p.cols - c));
    const bool in = inside(c, p.cols);
    unpack(load16(static_cast<const T *>(p.dy) + row * p.lddy + c, n, level(vec, 0), in), x.dy);
    if (p.dh) {
      unpack(load16(static_cast<const T *>(p.dh) + row * p.lddh + c, n, level(vec, 1), in), x.dh);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.dh[i] = both(0.0f);
    }
    const auto matrix = [&](const Kept &k, int lv, float2 (&v)[8]) {
      if (k.s)
        unpack_kept<3>(load16_fp8(static_cast<const unsigned char *>(k.p) + row * k.ld + c, n, lv), k.s[row * k.lds + (c >> 7)],
                    k.e5m2, v);
      else
        unpack(load16(static_cast<const T *>(k.p) + row * k.ld + c, n, lv, in), v);
    };
    matrix(p.a, level(vec, 7), x.a);
    matrix(p.h, level(vec, 8), x.h);
    clear_kept(x, n);
    load16_w<T>(p.w, p.w_f32, c, n, level(vec, 2), w);
    load_gated<T>(p, group, c, n, vec, m);
    return n;
  };
  for (unsigned row = r0; row < r1; ++row) {
    const float t = p.t[row], tp = p.tp[row];
    const unsigned group = p.gate.p ? row / p.gate.rows : 0;
    float total[4] = {};
    for (int64_t c = threadIdx.x * 16; c < p.cols; c += kLongElements) {
      load(row, group, c);
      add_sums(x, w, m, t, total[0], total[1], total[2]);
    }
    row_sums(total);
    const Factors f = factors(t, tp, total[0], total[1], total[2], mean);
    const bool begins = row == r0 || (p.gate.p && row % p.gate.rows == 0);
    const bool ends = row + 1 == r1 || (p.gate.p && (row + 1) % p.gate.rows == 0);
    for (int64_t c = threadIdx.x * 16; c < p.cols; c += kLongElements) {
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
        flush<T>(p, blockIdx.x, group, r0, r1, c, n, sn, first, vec);
      else
        store_part(part(p, blockIdx.x, kTail, c), sn);
    }
    if (ends) first = false;
  }
}

// Sums over clusters in a fixed order: blockIdx.y 0 of dw, 1 of dwp (and dgate, if it has one row), then of the gate rows
// that several clusters share, which are found by the gate row (by_group) or by the boundary between two clusters.  A CTA
// takes 32 columns, four a thread, and every 32nd cluster, eight loads in flight (with a column a thread, 1024 of them, and
// five loads 1024 clusters' rows of 1024 columns took 11.4 us, now 8.4).
template <class T>
__global__ void __launch_bounds__(256) sandwich_sums_kernel(const SandwichGradParams p, const Split split,
                                                            const bool by_group) {
  __shared__ float red[8][32];
  griddep_wait();
  unsigned first = 0, end = split.clusters, group = 0;
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
  } else if (blockIdx.y ? !p.dwp && !(p.dgate && one_gate(p)) : !p.dw) {
    return;
  }
  const auto kind = [&](unsigned b) {
    return blockIdx.y == 0   ? kDw
           : blockIdx.y == 1 ? kDwp
           : static_cast<int64_t>(group) * p.gate.rows < static_cast<int64_t>(b) * split.rows ? kHead
                                                                                              : kTail;
  };
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 7) * 4;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < p.cols) {   // (a part's row is a multiple of 16 long)
    for (unsigned b0 = first + (threadIdx.x >> 3); b0 < end; b0 += 256) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = b0 + 32 * i < end ? *reinterpret_cast<const float4 *>(part(p, b0 + 32 * i, kind(b0 + 32 * i), c))
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = make_float4(sum.x + v[i].x, sum.y + v[i].y, sum.z + v[i].z, sum.w + v[i].w);
    }
  }
#pragma unroll
  for (int d = 8; d <= 16; d <<= 1) {
    sum.x += __shfl_xor_sync(~0u, sum.x, d);
    sum.y += __shfl_xor_sync(~0u, sum.y, d);
    sum.z += __shfl_xor_sync(~0u, sum.z, d);
    sum.w += __shfl_xor_sync(~0u, sum.w, d);
  }
  if ((threadIdx.x & 31) < 8) {
    float *to = &red[threadIdx.x >> 5][(threadIdx.x & 7) * 4];
    to[0] = sum.x;
    to[1] = sum.y;
    to[2] = sum.z;
    to[3] = sum.w;
  }
  __syncthreads();
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || o >= p.cols) return;
  float total = red[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < 8; ++w) total += red[w][threadIdx.x];
  const auto value = [&](const void *w, bool f32) {
    return f32 ? static_cast<const float *>(w)[o] : to_float(static_cast<const T *>(w)[o]);
  };
  const auto put = [&](void *d, bool f32, int64_t at, float v) {
    if (f32)
      static_cast<float *>(d)[at] = v;
    else
      from_float(static_cast<T *>(d) + at, v);
  };
  if (blockIdx.y == 0) {
    put(p.dw, p.w_f32, o, total);
  } else if (blockIdx.y == 1) {
    if (p.dwp) put(p.dwp, p.w_f32, o, p.gate.p && one_gate(p) && p.rows > 0 ? value(p.gate.p, p.gate.f32) * total : total);
    if (p.dgate && one_gate(p)) put(p.dgate, p.gate.f32, o, value(p.wp, p.w_f32) * total);
  } else {
    put(p.dgate, p.gate.f32, group * p.lddgate + o, value(p.wp, p.w_f32) * total);
  }
}

// How rows are laid over threads and CTAs: 512 threads an SM.
struct RowsShape {
  int threads, per_sm;
  bool segments;
  Split split;
};
RowsShape rows_shape(int64_t rows, int64_t cols, int sm_count) {
  const int64_t chunks = (cols + 15) / 16;
  RowsShape g;
  g.segments = chunks > kMaxCluster * kClusterThreads;
  unsigned cluster = 1;
  while (!g.segments && chunks > cluster * kClusterThreads) cluster *= 2;
  g.threads = g.segments ? kLongThreads : static_cast<int>(((chunks + cluster - 1) / cluster + 31) / 32 * 32);
  g.per_sm = g.segments ? 1 : 512 / g.threads;
  // (clusters of four and eight find room on all but four of a GB300's SMs, whatever the CTAs an SM: with one cluster for
  // every four CTAs of all SMs the last ones ran by themselves, 8192 x 8192 with checkpoints 248 us)
  const int64_t most = static_cast<int64_t>(cluster >= 4 && sm_count > 8 ? sm_count - 4 : sm_count) * g.per_sm / cluster;
  const int64_t each = rows > 0 ? (rows + most - 1) / most : 1;
  g.split = {static_cast<unsigned>((rows + each - 1) / each), static_cast<unsigned>(each), cluster};
  return g;
}

template <class T, int KIND>
cudaError_t rows_kernel(const SandwichGradParams &p, const RowsShape &g, uint32_t vec, cudaStream_t s) {
  constexpr int bytes = RowPlaces<T, KIND>::kBytes;
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [dev] {
    set[dev] = cudaFuncSetAttribute(sandwich_backward_kernel<T, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    RowPlaces<T, KIND>::kBytes * kClusterThreads);
  });
  if (set[dev] != cudaSuccess) return set[dev];
  return launch_cluster_maybe_pdl(sandwich_backward_kernel<T, KIND>, dim3(g.split.clusters * g.split.cluster),
                                  dim3(g.threads), static_cast<size_t>(bytes) * g.threads, s, true,
                                  static_cast<int>(g.split.cluster), p, g.split, vec);
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
      err = launch_maybe_pdl(sandwich_backward_long_kernel<T>, dim3(g.split.clusters), dim3(g.threads), 0, s, true, p, g.split, vec);
    else if (!p.a.s != !p.h.s || p.a.e5m2 != p.h.e5m2)
      err = rows_kernel<T, 3>(p, g, vec, s);
    else if (!p.a.s)
      err = rows_kernel<T, 0>(p, g, vec, s);
    else
      err = p.a.e5m2 ? rows_kernel<T, 2>(p, g, vec, s) : rows_kernel<T, 1>(p, g, vec, s);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  if (!sums) return cudaSuccess;
  unsigned shared = 0;   // gate rows to be looked at
  bool by_group = false;
  if (p.dgate && p.rows > 0 && !one_gate(p) && g.split.rows % p.gate.rows != 0) {
    const int64_t groups = (p.rows + p.gate.rows - 1) / p.gate.rows;
    by_group = groups < g.split.clusters;
    shared = by_group ? static_cast<unsigned>(groups) : g.split.clusters - 1;
  }
  ++*launches;
  return launch_maybe_pdl(sandwich_sums_kernel<T>, dim3(static_cast<unsigned>((p.cols + 31) / 32), 2 + shared),
                          dim3(256), 0, s, true, p, g.split, by_group);
}

}  // namespace

int64_t sandwich_partials(int64_t rows, int64_t cols) {
  return static_cast<int64_t>(rows_shape(rows, cols, kSms).split.clusters) * kParts * part_pitch(cols);
}

cudaError_t launch_sandwich_norm_backward(const SandwichGradParams &p, cudaStream_t s, int *launches) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return typed<float>(p, s, launches);
    case SGEMM_TYPE_BF16: return typed<__nv_bfloat16>(p, s, launches);
    default: return typed<__half>(p, s, launches);
  }
}

}  // namespace sg
