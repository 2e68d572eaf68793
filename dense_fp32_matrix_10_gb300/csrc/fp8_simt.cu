// fp8_simt.cu -- the block-scaled 8-bit product on CUDA cores: any layout and
// alignment.  C = alpha * sum_b SA SB (sum_{k in b} A B) + beta * C.
//
// 64 x 64 outputs per CTA, 4 x 4 per thread; k in slices of 32 converted to
// FP32 in shared memory; the sum of a block of 128 is scaled and added to the
// output's sum when the block ends.
#include "fp8.cuh"
#include "fp8.h"
#include "internal.h"

namespace sg {
namespace {

constexpr int BM = 64, BN = 64, BK = 32, PITCH = BM + 4;

// The 64 x 32 slice of an operand at (o0, k0), k-major, as floats; element
// loads in the order of the stored layout, zeros outside.
__device__ __forceinline__ void load_slice(const Fp8Operand &x, int o0, int k0, int outer, int K,
                                           float (*dst)[PITCH]) {
#pragma unroll
  for (int i = 0; i < BM * BK / 256; ++i) {
    const int e = threadIdx.x + 256 * i;
    const int o = x.inner_rows ? e % BM : e / BK, k = x.inner_rows ? e / BM : e % BK;
    uint32_t b = 0;
    if (o0 + o < outer && k0 + k < K)
      b = x.q[x.inner_rows ? (k0 + k) * x.ld + (o0 + o) : (o0 + o) * x.ld + (k0 + k)];
    dst[k][o] = from_fp8x2(b, x.e5m2).x;
  }
}

__device__ __forceinline__ float scale_of(const Fp8Operand &x, int o, int outer, int kb) {
  if (o >= outer) return 0.0f;
  const int64_t i = o >> x.shift;
  return x.s[x.inner_rows ? kb * x.lds + i : i * x.lds + kb];
}

template <class T>
__device__ __forceinline__ void put(const Fp8Params &p, int m, int n, float v) {
  T *c = static_cast<T *>(p.C) + m * p.ldc + n;
  v *= p.alpha;
  if (p.beta != 0.0f) v += p.beta * to_float(*c);
  from_float(c, v);
}

template <class T>
__global__ void __launch_bounds__(256) fp8_simt_kernel(const Fp8Params p, const int tiles_n) {
  __shared__ __align__(16) float as[BK][PITCH], bs[BK][PITCH];
  griddep_wait();
  const int m0 = static_cast<int>(blockIdx.x / tiles_n) * BM, n0 = static_cast<int>(blockIdx.x % tiles_n) * BN;
  const int tm = threadIdx.x / 16 * 4, tn = threadIdx.x % 16 * 4;
  float acc[4][4] = {}, blk[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += BK) {
    __syncthreads();
    load_slice(p.a, m0, k0, p.M, p.K, as);
    load_slice(p.b, n0, k0, p.N, p.K, bs);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      const float4 a = *reinterpret_cast<const float4 *>(&as[k][tm]);
      const float4 b = *reinterpret_cast<const float4 *>(&bs[k][tn]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) blk[i][j] += av[i] * bv[j];
    }
    if ((k0 + BK) % SGEMM_FP8_BLOCK == 0 || k0 + BK >= p.K) {
      const int kb = k0 / SGEMM_FP8_BLOCK;
      float sa[4], sb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sa[i] = scale_of(p.a, m0 + tm + i, p.M, kb);
        sb[i] = scale_of(p.b, n0 + tn + i, p.N, kb);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] += blk[i][j] * sb[j] * sa[i];
          blk[i][j] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (m0 + tm + i < p.M && n0 + tn + j < p.N) put<T>(p, m0 + tm + i, n0 + tn + j, acc[i][j]);
}

template <class T>
__global__ void __launch_bounds__(256) fp8_scale_c_kernel(const Fp8Params p) {
  griddep_wait();
  const int64_t total = static_cast<int64_t>(p.M) * p.N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    T *c = static_cast<T *>(p.C) + i / p.N * p.ldc + i % p.N;
    from_float(c, p.beta != 0.0f ? p.beta * to_float(*c) : 0.0f);
  }
}

template <class F>
cudaError_t by_type(int type, F f) {
  switch (type) {
    case SGEMM_TYPE_F32: return f(float());
    case SGEMM_TYPE_BF16: return f(__nv_bfloat16());
    default: return f(__half());
  }
}

}  // namespace

cudaError_t launch_fp8_simt(const Fp8Params &p, cudaStream_t s) {
  const int64_t tn = (static_cast<int64_t>(p.N) + BN - 1) / BN, tm = (static_cast<int64_t>(p.M) + BM - 1) / BM;
  if (tn * tm > 0x7fffffff) return cudaErrorInvalidValue;
  return by_type(p.typeC, [&](auto t) {
    return launch_maybe_pdl(fp8_simt_kernel<decltype(t)>, dim3(static_cast<unsigned>(tn * tm)), dim3(256), 0, s,
                            true, p, static_cast<int>(tn));
  });
}

cudaError_t launch_fp8_scale_c(const Fp8Params &p, cudaStream_t s) {
  const int64_t blocks = (static_cast<int64_t>(p.M) * p.N + 1023) / 1024;
  return by_type(p.typeC, [&](auto t) {
    return launch_maybe_pdl(fp8_scale_c_kernel<decltype(t)>, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)),
                            dim3(256), 0, s, true, p);
  });
}

}  // namespace sg
