// swiglu_backward.cuh -- the gradient of the gated unit as operands of the
// products that follow:
//
//   du = dy g p,   dg = dy u p (1 + g (1 - p)),   y = g p u,   p = 1 / (1 + exp(-g))
//
// dg and du in 1 x 128 and in 128 x 1 blocks, y in 128 x 1 blocks: a CTA takes
// a 128 x 128 tile at a time, so that every block of either orientation lies
// in one CTA.  Eight lanes hold a row of it, a thread 2 x 16 elements, whose
// 96 values stay in FP32 registers from the maxima to the quotients.  That
// leaves room for one CTA of 512 threads an SM: it walks over tiles, and a
// thread copies its elements of the next tile to places of its own in shared
// memory while it quantises this one.  4095 x 8192 bf16 from checkpoints 85 us,
// 3.6 TB/s, 45 instructions an element at 48 % of the issue slots (16 warps).
#pragma once

#include <mutex>

#include "dispatch.h"
#include "swiglu.cuh"

namespace sg {

constexpr int kUnitThreads = 512;

// SRC: g and u are 0 matrices of T, 1 checkpoints in E4M3, 2 in E5M2.
template <class T, int SRC>
struct UnitTile {
  static constexpr int kDy = sizeof(T), kG = SRC ? 1 : sizeof(T);   // 16-byte units of 16 elements
  static constexpr int kUnits = kDy + 2 * kG;                       // of a row's 16 elements
  static constexpr int kMine = 2 * kUnits + (SRC ? 1 : 0);          // of a thread: two rows', and the scales of their g, u
  static constexpr int kRaw = kMine * kUnitThreads * 16;
  static constexpr int kPart = 16 * 3 * 128 * 4, kInv = 3 * 128 * 4;
  static constexpr int kBytes = kRaw + kPart + kInv;
};

// RAGGED: a row's last block has zeros behind the row's end.  A block with a NaN or an infinity would make NaN of them, when
// the zeros of a checkpoint meet its scale and when its own zeros are quantised (4000 x 4001 bf16 from checkpoints 53.9 us,
// without looking after them 52.4; where no row ends inside a block that would cost 4095 x 8192 88 us instead of 85).
// vec: 0 dy, 1 g, 2 u, 3 qr, 4 qc, 5 qy
template <class T, int SRC, bool Z_E5M2, bool RAGGED>
__global__ void __launch_bounds__(kUnitThreads, 1)
    swiglu_backward_kernel(const SwigluGradParams p, const unsigned tiles_c, const unsigned tiles, const uint32_t vec) {
  using Tile = UnitTile<T, SRC>;
  extern __shared__ __align__(16) unsigned char smem[];
  uint4 *raw = reinterpret_cast<uint4 *>(smem) + first_unit(Tile::kMine);      // [2][dy, g, u]
  float *src_scale = reinterpret_cast<float *>(raw + 2 * Tile::kUnits * kUnitStep);   // [2][g, u]
  float *part = reinterpret_cast<float *>(smem + Tile::kRaw);                  // [warp][dg, du, y][column] maxima
  float *col_inv = reinterpret_cast<float *>(smem + Tile::kRaw + Tile::kPart);    // [3][column_place()] -1 / scale
  griddep_wait();
  griddep_launch_dependents();
  const int lane8 = threadIdx.x & 7, row64 = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int64_t wide = static_cast<int64_t>(tiles_c) * 128;

  // (a tile's offsets are the same for the whole CTA, so that only the thread's own are left to each)
  const auto fetch = [&](unsigned tile) {
    const unsigned tr = tile / tiles_c, tc = tile - tr * tiles_c;
    const int64_t top = static_cast<int64_t>(tr) * 128, left = static_cast<int64_t>(tc) * 128;
    const int n = static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - left - lane8 * 16)));
    const int rows = static_cast<int>(min(int64_t(128), p.rows - top));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 64 * i + row64, m = row < rows ? n : 0;
      const auto matrix = [&](const void *base, int64_t ld, int lv, uint4 *to) {
        copy16(to, static_cast<const T *>(base) + top * ld + left + row * ld + lane8 * 16, m, lv,
               m == 16 && inside(left + lane8 * 16, p.cols));
      };
      uint4 *to = raw + i * Tile::kUnits * kUnitStep;
      matrix(p.dy, p.lddy, level(vec, 0), to);
      to += Tile::kDy * kUnitStep;
      if constexpr (SRC != 0) {
        const auto kept = [&](const Kept &k, int lv, uint4 *place, float *scale) {
          copy16_kept(place, scale, static_cast<const unsigned char *>(k.p) + top * k.ld + left + row * k.ld + lane8 * 16,
                      k.s + top * k.lds + tc + row * k.lds, m, lv);
        };
        kept(p.g, level(vec, 1), to, src_scale + 2 * i);
        kept(p.u, level(vec, 2), to + kUnitStep, src_scale + 2 * i + 1);
      } else {
        matrix(p.g.p, p.g.ld, level(vec, 1), to);
        matrix(p.u.p, p.u.ld, level(vec, 2), to + Tile::kDy * kUnitStep);
      }
    }
    copies_commit();
  };
  const auto take = [&](const uint4 *at, float2 (&x)[8]) { unpack(take16<T>(at), x); };
  const auto take_kept = [&](const uint4 *at, float scale, int n, float2 (&x)[8]) {
    unpack_fp8<SRC == 2>(*at, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], both(scale));
    if (RAGGED) clear_from(x, n);
  };

  fetch(blockIdx.x);
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const unsigned tr = tile / tiles_c, tc = tile - tr * tiles_c;
    const int64_t top = static_cast<int64_t>(tr) * 128, left = static_cast<int64_t>(tc) * 128;
    const int n = static_cast<int>(max(int64_t(0), min(int64_t(16), p.cols - left - lane8 * 16)));
    const int rows = static_cast<int>(min(int64_t(128), p.rows - top));
    const bool live[2] = {row64 < rows, row64 + 64 < rows};
    float2 v[3][2][8];   // -dg, -du, -y
    copies_wait(0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 *at = raw + i * Tile::kUnits * kUnitStep;
      float2 dy[8], g[8], u[8];
      take(at, dy);
      at += Tile::kDy * kUnitStep;
      if constexpr (SRC != 0) {
        take_kept(at, src_scale[2 * i], n, g);
        take_kept(at + kUnitStep, src_scale[2 * i + 1], n, u);
      } else {
        take(at, g);
        take(at + Tile::kDy * kUnitStep, u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 np = negated_logistic(g[j]), ngp = mul2(g[j], np);                // -p, -g p
        const float2 nslope = fma2(ngp, add2(np, both(1.0f)), np);               // -(p + g p (1 - p))
        v[0][i][j] = mul2(mul2(dy[j], u[j]), nslope);
        v[1][i][j] = mul2(dy[j], ngp);
        v[2][i][j] = mul2(ngp, u[j]);
      }
    }
    if (tile + gridDim.x < tiles) fetch(tile + gridDim.x);
    // the column maxima of the warp's eight rows: a lane keeps the half of its columns that it owns, then half of those
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const bool h16 = threadIdx.x & 16, h8 = threadIdx.x & 8;
      float2 a[4], b[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 lo = make_float2(max_abs(v[k][0][j].x, v[k][1][j].x), max_abs(v[k][0][j].y, v[k][1][j].y));
        const float2 hi = make_float2(max_abs(v[k][0][4 + j].x, v[k][1][4 + j].x), max_abs(v[k][0][4 + j].y, v[k][1][4 + j].y));
        const float2 mine = h16 ? hi : lo, give = h16 ? lo : hi;
        a[j] = make_float2(max_abs(mine.x, __shfl_xor_sync(~0u, give.x, 16)), max_abs(mine.y, __shfl_xor_sync(~0u, give.y, 16)));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 mine = h8 ? a[2 + j] : a[j], give = h8 ? a[j] : a[2 + j];
        b[j] = make_float2(max_abs(mine.x, __shfl_xor_sync(~0u, give.x, 8)), max_abs(mine.y, __shfl_xor_sync(~0u, give.y, 8)));
      }
      *reinterpret_cast<float4 *>(part + (warp * 3 + k) * 128 + lane8 * 16 + (h16 ? 8 : 0) + (h8 ? 4 : 0)) =
          make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
    }
    __syncthreads();
    if (threadIdx.x < 384) {
      const unsigned kind = threadIdx.x >> 7, col = threadIdx.x & 127;
      float a = part[kind * 128 + col];
#pragma unroll
      for (int w = 1; w < 15; w += 2) a = max_abs3(a, part[(w * 3 + kind) * 128 + col], part[((w + 1) * 3 + kind) * 128 + col]);
      a = max_abs(a, part[(15 * 3 + kind) * 128 + col]);
      const float s = scale_of(a, kind == 2 ? p.y_e5m2 : Z_E5M2);
      col_inv[kind * 128 + column_place(col)] = -inv_of(s);
      const int64_t at = left + col;
      if (kind < 2)
        p.sc[tr * p.ldsc + kind * wide + at] = s;
      else if (at < p.cols)
        p.sy[tr * p.ldsy + at] = s;
    }
    // meanwhile the row blocks of dg and du: four maxima over eight lanes
    {
      const float m[4] = {max_abs16(v[0][0]), max_abs16(v[0][1]), max_abs16(v[1][0]), max_abs16(v[1][1])};
      const int own = owned_by(lane8);
      const float s = scale_of(owned_max(m, lane8), Z_E5M2), ninv = -inv_of(s);
      const int mine = row64 + 64 * (own & 1);
      if ((lane8 & 1) == 0 && mine < rows) (p.sr + top * p.ldsr + tc)[mine * p.ldsr + (own >> 1) * tiles_c] = s;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        unsigned char *q = p.qr + top * p.ldqr + k * wide + left + row64 * p.ldqr + lane8 * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float r = __shfl_sync(~0u, ninv, owner_of(2 * k + i), 8);
          uint4 z = quantise<Z_E5M2>(v[k][i], r);
          if (RAGGED) z = first16_fp8(z, n);
          if (live[i]) store16_fp8(q + 64 * i * p.ldqr, z, 16, level(vec, 3));
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int64_t ld = k < 2 ? p.ldqc : p.ldqy;
      unsigned char *q = (k < 2 ? p.qc + k * wide : p.qy) + top * ld + left + row64 * ld + lane8 * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 r = column_values(col_inv + k * 128, lane8, j);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v[k][i][2 * j] = mul2(v[k][i][2 * j], make_float2(r.x, r.y));
          v[k][i][2 * j + 1] = mul2(v[k][i][2 * j + 1], make_float2(r.z, r.w));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!live[i]) continue;
        if (k < 2)
          store16_fp8(q + 64 * i * ld, to_fp8x16<Z_E5M2>(v[k][i]), 16, level(vec, 4));
        else
          store16_fp8(q + 64 * i * ld, p.y_e5m2 ? to_fp8x16<true>(v[k][i]) : to_fp8x16<false>(v[k][i]), n, level(vec, 5));
      }
    }
  }
}

template <class T, int SRC, bool Z_E5M2, bool RAGGED>
cudaError_t launch_unit_gradient_of(const SwigluGradParams &p, int sm_count, cudaStream_t s) {
  const int64_t tiles_c = (p.cols + 127) / 128, tiles = tiles_c * ((p.rows + 127) / 128);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  static std::once_flag once[kMaxDevices];
  static cudaError_t set[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  constexpr int bytes = UnitTile<T, SRC>::kBytes;
  std::call_once(once[dev], [dev] {
    set[dev] = cudaFuncSetAttribute(swiglu_backward_kernel<T, SRC, Z_E5M2, RAGGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    UnitTile<T, SRC>::kBytes);
  });
  if (set[dev] != cudaSuccess) return set[dev];
  constexpr int e = sizeof(T), ek = SRC ? 1 : e;
  const uint32_t vec = level_of(p.dy, p.lddy, e, 0) | level_of(p.g.p, p.g.ld, ek, 1) | level_of(p.u.p, p.u.ld, ek, 2) |
                       level_of(p.qr, p.ldqr, 1, 3) | level_of(p.qc, p.ldqc, 1, 4) | level_of(p.qy, p.ldqy, 1, 5);
  const unsigned grid = static_cast<unsigned>(tiles < sm_count ? tiles : sm_count);
  return launch_maybe_pdl(swiglu_backward_kernel<T, SRC, Z_E5M2, RAGGED>, dim3(grid), dim3(kUnitThreads), bytes, s, true, p,
                          static_cast<unsigned>(tiles_c), static_cast<unsigned>(tiles), vec);
}

template <class T, int SRC, bool Z_E5M2>
cudaError_t launch_unit_gradient(const SwigluGradParams &p, int sm_count, cudaStream_t s) {
  return p.cols % 128 ? launch_unit_gradient_of<T, SRC, Z_E5M2, true>(p, sm_count, s)
                      : launch_unit_gradient_of<T, SRC, Z_E5M2, false>(p, sm_count, s);
}

template <class T>
cudaError_t launch_unit_gradient(const SwigluGradParams &p, int sm_count, cudaStream_t s) {
  const auto of = [&](auto e4m3, auto e5m2) { return p.z_e5m2 ? e5m2(p, sm_count, s) : e4m3(p, sm_count, s); };
  if (!p.g.s) return of(launch_unit_gradient<T, 0, false>, launch_unit_gradient<T, 0, true>);
  if (p.g.e5m2) return of(launch_unit_gradient<T, 2, false>, launch_unit_gradient<T, 2, true>);
  return of(launch_unit_gradient<T, 1, false>, launch_unit_gradient<T, 1, true>);
}

}  // namespace sg
