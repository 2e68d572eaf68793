// swiglu.cu -- the gated unit y = g p u, p = 1 / (1 + exp(-g)), with a
// quantised output, one 1 x 128 block by eight lanes, 16 elements a lane and
// nothing between CTAs: 33 instructions an element with checkpoints, 18 without,
// are near memory's rate (8192 x 8192 bf16 84 us, 5.6 TB/s, and 57 us, 5.9 TB/s).
#include "dispatch.h"
#include "fp8_block.cuh"
#include "swiglu.cuh"

namespace sg {
namespace {

// KEEP: 0 no checkpoints, 1 in E4M3, 2 in E5M2 (of either or both).  vec: 0 g, 1 u, 2 q, 3 qg, 4 qu.
template <class T, bool E5M2, int KEEP>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3)
    swiglu_kernel(const SwigluParams p, const unsigned blocks_c, const int64_t units, const uint32_t vec) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane8 = threadIdx.x & 7;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 3);
  // (a division in 64 bits takes some 100 instructions, in 32 bits 15)
  const int64_t row = units <= 0xffffffe0ll ? static_cast<unsigned>(unit) / blocks_c : unit / blocks_c;
  const unsigned block = static_cast<unsigned>(unit - row * blocks_c);
  const int64_t c = static_cast<int64_t>(block) * 128 + lane8 * 16;
  const int n = unit < units ? static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - c))) : 0;
  // with checkpoints g and u have the other sign, which the exact quotients want
  const bool in = n == 16 && inside(c, p.cols);
  Raw16<T> rg = load16(static_cast<const T *>(p.g) + row * p.ldg + c, n, level(vec, 0), in);
  Raw16<T> ru = load16(static_cast<const T *>(p.u) + row * p.ldu + c, n, level(vec, 1), in);
  if (KEEP) {
    rg = negated(rg);
    ru = negated(ru);
  }
  float2 y[8], g[8], u[8];
  unpack(rg, g);
  unpack(ru, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 np = negated_logistic(KEEP ? make_float2(-g[i].x, -g[i].y) : g[i]);
    y[i] = mul2(mul2(g[i], np), u[i]);   // -y; with checkpoints -g, -u and so -y, too
  }
  float scale;
  int own = 0;
  if (KEEP) {
    const float m[4] = {max_abs16(y), max_abs16(g), max_abs16(u), 0.0f};
    own = owned_by(lane8);
    scale = scale_of(owned_max(m, lane8), own == 0 ? E5M2 : KEEP == 2);
  } else {
    scale = scale_of(max_of_8(max_abs16(y)), E5M2);
  }
  const auto of = [&](float v, int i) { return KEEP ? __shfl_sync(~0u, v, owner_of(i), 8) : v; };
  store16_fp8(p.q + row * p.ldq + c, quantise<E5M2>(y, -of(inv_of(scale), 0)), n, level(vec, 2));
  if (lane8 == owner_of(0) && n > 0) p.s[row * p.lds + block] = scale;
  if (KEEP) {
    const float div = divisor(scale), ninv = ninv_of(scale);
    const float dg = of(div, 1), ng = of(ninv, 1), du = of(div, 2), nu = of(ninv, 2);
    if (p.qg) {
      store16_fp8(p.qg + row * p.ldqg + c, quantise_exactly<KEEP == 2>(g, dg, ng), n, level(vec, 3));
      if (lane8 == owner_of(1) && unit < units) p.sg[row * p.ldsg + block] = scale;
    }
    if (p.qu) {
      store16_fp8(p.qu + row * p.ldqu + c, quantise_exactly<KEEP == 2>(u, du, nu), n, level(vec, 4));
      if (lane8 == owner_of(2) && unit < units) p.su[row * p.ldsu + block] = scale;
    }
  }
}

template <class T, bool E5M2>
cudaError_t typed(const SwigluParams &p, cudaStream_t s) {
  const int64_t blocks_c = (p.cols + 127) / 128, units = blocks_c * p.rows, ctas = (units + 31) / 32;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  constexpr int e = sizeof(T);
  const uint32_t vec = level_of(p.g, p.ldg, e, 0) | level_of(p.u, p.ldu, e, 1) | level_of(p.q, p.ldq, 1, 2) |
                       level_of(p.qg, p.ldqg, 1, 3) | level_of(p.qu, p.ldqu, 1, 4);
  const auto kernel = !(p.qg || p.qu) ? swiglu_kernel<T, E5M2, 0> : p.keep_e5m2 ? swiglu_kernel<T, E5M2, 2> : swiglu_kernel<T, E5M2, 1>;
  return launch_maybe_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, true, p,
                          static_cast<unsigned>(blocks_c), units, vec);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluParams &p, cudaStream_t s) {
  switch (p.typeX) {
    case SGEMM_TYPE_F32: return p.e5m2 ? typed<float, true>(p, s) : typed<float, false>(p, s);
    case SGEMM_TYPE_BF16: return p.e5m2 ? typed<__nv_bfloat16, true>(p, s) : typed<__nv_bfloat16, false>(p, s);
    default: return p.e5m2 ? typed<__half, true>(p, s) : typed<__half, false>(p, s);
  }
}

}  // namespace sg
