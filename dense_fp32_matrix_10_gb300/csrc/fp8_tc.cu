// fp8_tc.cu -- instances of the tensor-core 8-bit product, the choice between them and
// their launch.
#include "fp8_tc.cuh"

#include <cudaTypedefs.h>

#include <cstring>

#include "dispatch.h"

namespace sg {
namespace {

// Tensor map of a row-major matrix of `elem`-byte elements: boxes of 128 bytes x box_rows, 128-byte swizzle, zeros
// outside.
bool encode_map(CUtensorMap *m, const void *base, int elem, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  // a single row has no stride to respect
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows == 1 ? (cols * elem + 15) / 16 * 16 : ld * elem)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem), static_cast<cuuint32_t>(box_rows)}, estr[2] = {1, 1};
  return fn(m,
            elem == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
            : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16
                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct KernelInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int clusters = 0;   // pairs resident at once (GROUP == 2)
};

template <class Cfg>
cudaLaunchConfig_t launch_config(unsigned grid, int cluster, cudaStream_t s, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cfg::THREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cfg;
}

// Once per device: the kernel's shared memory, its register split, the pairs that fit.
template <class Cfg>
const KernelInfo *kernel_info() {
  static KernelInfo info[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  KernelInfo &i = info[dev];
  std::call_once(i.once, [&] {
    i.err = cudaFuncSetAttribute(fp8_tc_kernel<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    cudaFuncAttributes a;
    if (i.err == cudaSuccess) i.err = cudaFuncGetAttributes(&a, fp8_tc_kernel<Cfg>);
    // setmaxnreg.inc waits until the launch's registers cover the split
    if (i.err == cudaSuccess && Cfg::SPLIT_REGS && a.numRegs * Cfg::THREADS < Cfg::SPLIT_TOTAL)
      i.err = cudaErrorInvalidConfiguration;
    if (i.err == cudaSuccess && Cfg::GROUP == 2) {
      cudaLaunchAttribute attr[2];
      const cudaLaunchConfig_t cfg = launch_config<Cfg>(304, 2, nullptr, attr);
      i.err = cudaOccupancyMaxActiveClusters(&i.clusters, fp8_tc_kernel<Cfg>, &cfg);
      if (i.err == cudaSuccess && i.clusters < 1) i.err = cudaErrorInvalidConfiguration;
    }
    if (i.err != cudaSuccess) cudaGetLastError();
  });
  return i.err == cudaSuccess ? &i : nullptr;
}

int size_of(int type) { return type == SGEMM_TYPE_F32 ? 4 : 2; }

// `split`: CTAs per tile (GROUP == 1).
template <class Cfg>
cudaError_t launch(const Fp8Params &p, int split, cudaStream_t s) {
  const KernelInfo *info = kernel_info<Cfg>();
  if (!info) return cudaErrorInvalidConfiguration;
  const Fp8Operand &row = Cfg::SWAP ? p.b : p.a, &col = Cfg::SWAP ? p.a : p.b;
  Fp8TcParams t;
  t.rows = Cfg::SWAP ? p.N : p.M;
  t.cols = Cfg::SWAP ? p.M : p.N;
  t.row_q = row.q;
  t.col_q = col.q;
  t.row_qld = row.ld;
  t.col_qld = col.ld;
  t.k = p.K;
  CUtensorMap tm_row = {}, tm_col = {}, tm_c = {};
  const auto encode = [&](CUtensorMap *m, const Fp8Operand &x, int outer, int box) {
    return x.inner_rows ? encode_map(m, x.q, 1, p.K, outer, x.ld, 128) : encode_map(m, x.q, 1, outer, p.K, x.ld, box);
  };
  if (!Cfg::LOAD && (!encode(&tm_row, row, t.rows, 128) || !encode(&tm_col, col, t.cols, Cfg::BN / Cfg::GROUP)))
    return cudaErrorInvalidValue;
  if (Cfg::BULK && !encode_map(&tm_c, p.C, size_of(p.typeC), p.M, p.N, p.ldc, 32)) return cudaErrorInvalidValue;
  t.row_s = row.s;
  t.col_s = col.s;
  t.row_ld = row.lds;
  t.col_ld = col.lds;
  t.row_shift = row.shift;
  t.col_shift = col.shift;
  t.row_inner = row.inner_rows;
  t.col_inner = col.inner_rows;
  t.row_vec = !row.inner_rows && aligned_rows(row.s, row.lds, 4, 16);
  t.kblocks = static_cast<int>((static_cast<int64_t>(p.K) + 127) / 128);
  const int64_t br = 128 * Cfg::GROUP;
  t.tiles_r = static_cast<int>((t.rows + br - 1) / br);
  t.tiles_c = static_cast<int>((static_cast<int64_t>(t.cols) + Cfg::BN - 1) / Cfg::BN);
  const int64_t tiles = static_cast<int64_t>(t.tiles_r) * t.tiles_c;
  if (tiles * split > 0x7fffffff) return cudaErrorInvalidValue;
  t.num_tiles = static_cast<int>(tiles);
  t.group = 8;
  t.split = split;
  t.idesc = idesc_fp8(128 * Cfg::GROUP, Cfg::BN, row.e5m2, col.e5m2, row.inner_rows, col.inner_rows);
  t.C = p.C;
  t.ldc = p.ldc;
  t.typeC = p.typeC;
  t.vecC = aligned_rows(p.C, p.ldc, size_of(p.typeC), 16);
  t.alpha = p.alpha;
  t.beta = p.beta;
  t.wait_budget_ns = p.wait_budget_ns;
  t.status = p.status;
  const int cluster = Cfg::GROUP == 2 ? 2 : split;
  const int64_t grid = Cfg::GROUP == 2 ? 2 * (tiles < info->clusters ? tiles : info->clusters) : tiles * split;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = launch_config<Cfg>(static_cast<unsigned>(grid), cluster, s, attr);
  return cudaLaunchKernelEx(&cfg, fp8_tc_kernel<Cfg>, tm_row, tm_col, tm_c, t);
}

using Pair = Fp8Tc<2, 256, false, false, 6, 1>;      // 256 x 256 on two SMs
using PairBulk = Fp8Tc<2, 256, false, false, 4, 1, false, false, true>;   // the same for a C that TMA can write
using PairStaged = Fp8Tc<2, 256, false, false, 5, 1, true>;   // the same for an unaligned C
using PairVec = Fp8Tc<2, 256, false, true, 6, 1, false>;
using PairVecBulk = Fp8Tc<2, 256, false, true, 4, 1, false, false, true>;
using Tile = Fp8Tc<1, 128, false, false, 3, 2>;      // 128 x 128, two CTAs an SM
using TileVec = Fp8Tc<1, 128, false, true, 3, 2>;
using Half = Fp8Tc<1, 64, false, false, 3, 2>;       // 128 x 64
using HalfVec = Fp8Tc<1, 64, false, true, 3, 2>;
using Few16 = Fp8Tc<1, 16, true, true, 5, 2>;        // up to 16, 32, 64 rows of C (its columns are the
using Few32 = Fp8Tc<1, 32, true, true, 5, 2>;        // tile's rows)
using Few64 = Fp8Tc<1, 64, true, true, 4, 2>;

using Loaded = Fp8Tc<1, 128, false, false, 5, 1, true, true>;   // 128 x 128 of operands that TMA cannot read
using LoadedVec = Fp8Tc<1, 128, false, true, 5, 1, true, true>;

// 16-byte aligned rows that a tensor map can describe.
bool tma_readable(const Fp8Operand &x, int64_t stored_rows) {
  return reinterpret_cast<uintptr_t>(x.q) % 16 == 0 && (stored_rows == 1 || (x.ld % 16 == 0 && x.ld < kMaxLd));
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Cycles that a product of `tiles` tiles of 128 x cols takes with `split` CTAs a tile, two CTAs an SM, as
// measured: 960 for a block of k of either width (1150 with a scale per column), 4000 for a CTA's first copies
// and its stores (more where C's rows are unaligned), and the exchange of partial tiles.
int64_t tile_cycles(int64_t tiles, int64_t kblocks, int cols, int split, int64_t slots, bool vec, bool aligned) {
  const int64_t store = split > 1 ? 1500 + 40 * cols : aligned ? 0 : 40 * cols;
  return cdiv64(tiles * split, slots) * (cdiv64(kblocks, split) * (vec ? 1150 : 960) + 4000 + store);
}
// The same of the forms for few rows of C, which the weights' way from memory bounds: a block takes 700
// cycles, or 560 a CTA where two share an SM.
int64_t few_cycles(int64_t tiles, int64_t kblocks, int cols, int split, int64_t sms) {
  const int64_t per_sm = cdiv64(tiles * split, sms);
  return per_sm * (cdiv64(kblocks, split) * (per_sm > 1 ? 560 : 700) + 1500) +
         (split > 1 ? 1500 + 20 * split * cols : 0);
}
// The split of at most `most` that makes `cycles(split)` least and leaves each CTA two blocks or more.
template <class F>
int pick_split(int64_t kblocks, int most, F cycles) {
  int best = 1;
  for (int split = 2; split <= most && kblocks >= 2 * split; split *= 2)
    if (cycles(split) < cycles(best)) best = split;
  return best;
}

}  // namespace

Fp8Choice choose_fp8_form(const Fp8Params &p, int sm_count) {
  const int64_t kb = cdiv64(p.K, 128), slots = 2 * sm_count;
  const bool readable =
      tma_readable(p.a, p.a.inner_rows ? p.K : p.M) && tma_readable(p.b, p.b.inner_rows ? p.K : p.N);
  if (p.M <= 64 && !p.a.inner_rows && readable) {
    const int cols = p.M <= 16 ? 16 : p.M <= 32 ? 32 : 64;
    const int split =
        pick_split(kb, 8, [&](int n) { return few_cycles(cdiv64(p.N, 128), kb, cols, n, sm_count); });
    return {cols == 16 ? SGEMM_FP8_FORM_FEW_16 : cols == 32 ? SGEMM_FP8_FORM_FEW_32 : SGEMM_FP8_FORM_FEW_64, split};
  }
  const bool vec = p.b.shift == 0, aligned = aligned_rows(p.C, p.ldc, size_of(p.typeC), 16);
  const int64_t rows = cdiv64(p.M, 128);
  // (clusters of eight were never the best: 100 x 4096 x 4096 9.7 us with four, 16.0 with eight)
  const auto tiles = [&](int n) { return tile_cycles(rows * cdiv64(p.N, 128), kb, 128, n, slots, vec, aligned); };
  const auto halves = [&](int n) { return tile_cycles(rows * cdiv64(p.N, 64), kb, 64, n, slots, vec, aligned); };
  if (!readable) {   // one CTA an SM, and about three times the cycles for a block (361 us at 4096^3)
    const int n = pick_split(kb, 4, [&](int n) {
      return tile_cycles(rows * cdiv64(p.N, 128), 3 * kb, 128, n, sm_count, false, aligned);
    });
    return {SGEMM_FP8_FORM_LOADED, n};
  }
  const int split = pick_split(kb, 4, tiles), split_half = pick_split(kb, 4, halves);
  const int64_t tile = tiles(split), half = halves(split_half);
  // a pair of SMs takes as long for a block of its 256 x 256 tile as two CTAs for one of theirs each; 3000 cycles
  // for a tile's first copies and its stores, more where its threads write unaligned rows.  (Of 37 calls in two
  // layouts 35 choices are within 5 % of the fastest form and split; 1000 x 1013 x 997 is 8 % off, 100 x 4096 x 4096
  // with a scale per column 14 %.)
  const int64_t pair =
      1500 + cdiv64(cdiv64(p.M, 256) * cdiv64(p.N, 256), sm_count / 2) * (kb * 920 + (aligned ? 3000 : 8000));
  if (pair <= tile && pair <= half) {
    // (a TMA store writes whole 16 bytes at the end of a row)
    const int size = size_of(p.typeC);
    const bool bulk = aligned && p.beta == 0.0f && static_cast<int64_t>(p.N) * size % 16 == 0 && p.ldc < kMaxLd / size;
    if (bulk) return {SGEMM_FP8_FORM_PAIR_BULK, 1};
    return {aligned || vec ? SGEMM_FP8_FORM_PAIR : SGEMM_FP8_FORM_PAIR_STAGED, 1};
  }
  if (half < tile) return {SGEMM_FP8_FORM_HALF, split_half};
  return {SGEMM_FP8_FORM_TILE, split};
}

cudaError_t launch_fp8_product(const Fp8Params &p, int sm_count, cudaStream_t s) {
  const Fp8Choice c = choose_fp8_form(p, sm_count);
  const bool vec = p.b.shift == 0;
  switch (c.form) {
    case SGEMM_FP8_FORM_FEW_16: return launch<Few16>(p, c.split, s);
    case SGEMM_FP8_FORM_FEW_32: return launch<Few32>(p, c.split, s);
    case SGEMM_FP8_FORM_FEW_64: return launch<Few64>(p, c.split, s);
    case SGEMM_FP8_FORM_HALF: return vec ? launch<HalfVec>(p, c.split, s) : launch<Half>(p, c.split, s);
    case SGEMM_FP8_FORM_TILE: return vec ? launch<TileVec>(p, c.split, s) : launch<Tile>(p, c.split, s);
    case SGEMM_FP8_FORM_LOADED: return vec ? launch<LoadedVec>(p, c.split, s) : launch<Loaded>(p, c.split, s);
    case SGEMM_FP8_FORM_PAIR: return vec ? launch<PairVec>(p, 1, s) : launch<Pair>(p, 1, s);
    case SGEMM_FP8_FORM_PAIR_STAGED: return launch<PairStaged>(p, 1, s);
    case SGEMM_FP8_FORM_PAIR_BULK: return vec ? launch<PairVecBulk>(p, 1, s) : launch<PairBulk>(p, 1, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace sg
