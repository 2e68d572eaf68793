// fp8_tc.cuh -- the block-scaled 8-bit product on the 5th-generation tensor
// cores (tcgen05, kind::f8f6f4, FP32 accumulators in tensor memory).
//
//   C[m,n] = alpha * sum_b SA(m,b) SB(n,b) * (sum_{k in block b} A(m,k) B(k,n)) + beta * C[m,n]
//
// A stage holds one block of 128 k of both operands: 128 bytes, one row of the
// 128-byte swizzle, in either orientation (k-contiguous rows, or outer-contiguous
// rows of a k-major slice: the MMA reads both).  Four MMAs of k = 32 sum a block
// into a fresh accumulator in tensor memory; the epilogue warps scale it and add
// it to FP32 registers while the next blocks are multiplied, so the tensor cores'
// truncating accumulator never holds more than 128 products and every scale is
// applied in FP32.
//
// The two scales of a block are multiplied before its sum is there, one multiplication for 128 columns (or, VEC, one
// a value beside the tensor memory's loads).  Their product may leave FP32's normal range where the scaled sum does
// not; the interface states what that costs.  Scaling the sum twice would be a second multiplication for every value
// in all forms, and a test for the rare case would take its slow way at every padded row (least scale).
//
// The tile's rows (tensor memory lanes, one per thread) come from the operand
// `row`, its columns from `col`.  A row's scale is one value per thread and block;
// a column's scale is one value for 128 columns, or one each (VEC).
//
// Roles (per CTA):
//   warp 0   TMA producer (one thread)
//   warp 1   tensor memory; in the (even) CTA one thread issues the MMAs
//   warp 2   VEC: copies the scales of four blocks at a time into a ring in shared memory
//            (cp.async: any stride, zeros past the edge)
//   warp 3   idle
//   warps 4+ epilogue; warp 4 + q + 4 h owns rows 32 q .. +31 and the h-th ECOLS columns
//   LOAD: four more warps in the place of the producer
// Every wait on an mbarrier is bounded; after giving up, a role lets its copies and
// MMAs land (bounded) and goes to the barriers at the end.
//
// What bounds the pairs (256 x 256 on two SMs, the form of large products): an accumulator of 256
// columns is handed to the epilogue and back while the only other one is filled, about 450 ns a
// block of k, where the MMAs alone take 320; and the 1400 W of the card, reached in sustained runs of
// 8192^3 (2.5 PFLOP/s, 448 us; 401 in short ones).  Tried, at 4096 x 4096 x 16384 in 245 us then: four
// accumulators of 128 columns (345), sixteen epilogue
// warps of 64 columns (285), the row scales through shared memory (279), four at a time (258).
// Single CTAs (128 x 128 or 128 x 64, two an SM) are bound the same way (512 x 4096 x 8192 25.2 us, without
// any copies 22.8), the few-token forms by their weights' way from memory and by latencies.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "fp8.cuh"
#include "fp8.h"
#include "ptx.cuh"
#include "simt_gemm.cuh"   // tile_coords

namespace sg {

struct Fp8TcParams {
  const unsigned char *row_q, *col_q;   // operands as stored and their row strides (LOAD)
  int64_t row_qld, col_qld;
  int k;
  const float *row_s, *col_s;         // scales
  int64_t row_ld, col_ld;             // their row strides
  int row_shift, col_shift;           // outer index >> shift = scale index
  int row_inner, col_inner;           // the scales (and the operand) have k along their rows
  int row_vec;                        // four consecutive blocks' row scales are an aligned vector
  int rows, cols, kblocks;            // extents of the two outer dimensions, blocks of k
  int tiles_r, tiles_c, num_tiles, group;
  int split;                          // CTAs of a cluster that share a tile's blocks (GROUP == 1)
  uint32_t idesc;
  void *C;
  int64_t ldc;
  int typeC, vecC;
  float alpha, beta;
  uint64_t wait_budget_ns;
  int *status;
};

// GROUP 2: a pair of CTAs computes 256 x BN (cta_group::2), each holding 128 rows and
// half of the columns' operand.  SWAP: the tile's columns are C's rows.
// STAGED, BULK: see below.  LOAD: four more warps read operands that TMA cannot, of any base and stride.
template <int GROUP_, int BN_, bool SWAP_, bool VEC_, int STAGES_, int CTAS_, bool STAGED_ = GROUP_ == 1,
          bool LOAD_ = false, bool BULK_ = false>
struct Fp8Tc {
  static constexpr int GROUP = GROUP_, BN = BN_, STAGES = STAGES_, CTAS = CTAS_;
  static constexpr bool SWAP = SWAP_, VEC = VEC_, LOAD = LOAD_;
  static_assert(!LOAD || (GROUP == 1 && BN == 128), "loaded operands: 128 x 128 tiles of one CTA");
  // (a tile of 64 columns takes the room of 128: of an outer-contiguous operand whole 128-byte rows are
  // copied, and it uses one half of them)
  static constexpr bool HALF_ROWS = BN == 64 && !SWAP_;
  static constexpr int ROW_BYTES = 128 * 128, COL_BYTES = (HALF_ROWS ? 128 : BN / GROUP) * 128;
  static constexpr int STAGE_BYTES = ROW_BYTES + COL_BYTES;
  static constexpr int ACCS = BN >= 128 ? 2 : BN == 64 ? 4 : 8;   // accumulators
  static constexpr int TMEM_COLS = ACCS * BN;
  static constexpr int ECOLS = BN == 256 ? 128 : BN;   // columns a thread adds up
  static constexpr int EPI_WARPS = 4 * (BN / ECOLS);
  static constexpr int THREADS = 128 + 32 * EPI_WARPS + (LOAD ? 128 : 0);
  // FRAG: a thread holds 4 rows and every fourth pair of columns instead of one row, so it reads a
  // quarter of the column scales.  A shared memory read fills 128 bytes of registers a cycle however
  // many lanes share an address: 128 scales for each of 256 threads and block are 1024 cycles, more
  // than the block's MMAs take (4096 x 4096 x 16384: 448 us with one row a thread, 363 so).
  static constexpr bool FRAG = VEC && !SWAP && BN >= 128;
  static constexpr int CHUNK = ECOLS == 128 && !FRAG ? 32 : ECOLS >= 64 ? 16 : ECOLS / 2;   // columns of a tensor memory load
  static_assert(ECOLS / CHUNK % 2 == 0, "chunks alternate between two buffers across blocks");
  // VEC: ring of scales, SCALE_BLOCKS blocks of k a slot (one wait per slot, not per block): the rows'
  // [row][block], then the columns' [block][column]
  static constexpr int SCALE_SLOTS = VEC ? 3 : 0, SCALE_BLOCKS = 4;
  static constexpr int COL_SCALES = 128 * SCALE_BLOCKS;   // index of the first column scale
  static constexpr int SCALE_BYTES = 4 * (COL_SCALES + SCALE_BLOCKS * BN);
  static constexpr int SCALE_OFFSET = STAGES * STAGE_BYTES;
  // STAGED: rows of C may start off 16 bytes; a warp's finished 32 x 16 sums then pass through shared memory
  // and are written two rows at a time (by a thread per row a C of 1000 x 1013 took 39 us, so 12; aligned rows
  // are written faster by their threads, 16 bytes at a time).  Single CTAs use the stage ring for that.
  // Pairs have a place for it only in the form for unaligned C: the 20 KB cost the aligned one 3 us of 74
  // at 4096^3, as the L1 cache that holds the row scales shrinks.
  static constexpr bool STAGED = STAGED_ && !SWAP && !FRAG;
  // BULK (pairs; beta 0, rows of C of whole 16 bytes): a warp writes its 32 x 128 values, or 32 x 64 of F32 at a
  // time, to shared memory as swizzled boxes of 128-byte rows and leaves them to TMA stores while it goes on
  // to the next tile.  Written by the threads, a tile's stores hold its SMs up for 3 us (4096^3 in BF16
  // 73.1 us, so 64.3).
  static constexpr bool BULK = BULK_;
  static_assert(!BULK || (GROUP == 2 && !STAGED), "bulk stores: pairs");
  static constexpr int STORE_PITCH = 20, STORE_BYTES = BULK ? 2 * 32 * 128 : 32 * STORE_PITCH * 4;   // per warp
  static constexpr bool STORE_ROOM = GROUP == 2 && (STAGED || BULK);
  static constexpr int STORE_OFFSET = STORE_ROOM ? SCALE_OFFSET + SCALE_SLOTS * SCALE_BYTES : 0;
  static constexpr int BAR_OFFSET =
      SCALE_OFFSET + SCALE_SLOTS * SCALE_BYTES + (STORE_ROOM ? EPI_WARPS * STORE_BYTES : 0);
  static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 2 * SCALE_SLOTS + 1;
  static constexpr int SMEM_BYTES = BAR_OFFSET + NUM_BARS * 8 + 16 + 1024;
  static_assert(VEC || BN % 64 == 0, "a thread's columns lie in one block of 128");
  static_assert(SMEM_BYTES * CTAS + CTAS * 1024 <= 233472, "shared memory over the SM's limit");
  static_assert(TMEM_COLS * CTAS <= 512, "tensor memory over the SM's limit");
  // ECOLS = 128: 128 sums and two chunks of 32 in flight per epilogue thread
  static constexpr bool SPLIT_REGS = ECOLS == 128;
  static constexpr int REGS_WG0 = 40, REGS_EPI = BN == 256 ? 232 : 216;
  static constexpr int SPLIT_TOTAL =
      128 * REGS_WG0 + 32 * EPI_WARPS * REGS_EPI + (LOAD ? 128 * ((65536 / CTAS / THREADS) & ~7) : 0);
  static_assert(!SPLIT_REGS || SPLIT_TOTAL <= THREADS * ((65536 / CTAS / THREADS) & ~7),
                "register split exceeds the launch budget");
  // a cluster's partial tiles, in the stage ring: lines along C's rows ([row][column], SWAP [column][row]),
  // so that a warp's reads of another CTA's are whole stretches of 64 bytes and more (16 bytes here and
  // there: 4100 cycles for the exchange at 24 x 8192 x 4096, so 1700).  The [row][column] pitch is an odd number of
  // 16-byte units: eight rows written at once lie in eight different ones.
  static constexpr int PART_LINES = SWAP ? BN : 128, PART_PITCH = SWAP ? 128 : BN + 4;
  static_assert(GROUP == 2 || PART_LINES * PART_PITCH * 4 <= STAGES * STAGE_BYTES, "partial tile does not fit");
};

template <class Cfg>
struct Fp8Bars {
  uint32_t base;
  __device__ uint32_t full(uint32_t s) const { return base + 8 * s; }
  __device__ uint32_t empty(uint32_t s) const { return base + 8 * (Cfg::STAGES + s); }
  __device__ uint32_t acc_full(uint32_t b) const { return base + 8 * (2 * Cfg::STAGES + b); }
  __device__ uint32_t acc_empty(uint32_t b) const { return base + 8 * (2 * Cfg::STAGES + Cfg::ACCS + b); }
  __device__ uint32_t sc_full(uint32_t r) const { return base + 8 * (2 * Cfg::STAGES + 2 * Cfg::ACCS + r); }
  __device__ uint32_t sc_empty(uint32_t r) const {
    return base + 8 * (2 * Cfg::STAGES + 2 * Cfg::ACCS + Cfg::SCALE_SLOTS + r);
  }
  __device__ uint32_t drain() const { return base + 8 * (Cfg::NUM_BARS - 1); }
};

// D[tmem] (+)= A * B, kind::f8f6f4; one thread.
template <int GROUP>
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (GROUP == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shared-memory descriptor of a tile of 128-byte rows with the 128-byte swizzle, groups
// of 8 rows 1024 bytes apart.  k-contiguous: a row is one outer index, and 32 bytes
// further along it starts the next MMA's k.  Outer-contiguous: a row is one k of 128
// outer indices, and the next 32 k are 4096 bytes on; one swizzle atom spans all 128
// outer indices, so only the stride between groups of 8 k matters (given in both fields).
__device__ __forceinline__ uint64_t desc_fp8(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1024 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor: F32 accumulator, element types (0 E4M3, 1 E5M2), outer-contiguous
// operands (bits 15, 16), N and M.
inline uint32_t idesc_fp8(int M, int N, bool a_e5m2, bool b_e5m2, bool a_mn, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_e5m2) << 7) | (static_cast<uint32_t>(b_e5m2) << 10) |
         (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Wait for this thread's tensor memory loads; the values pass through, so that no use of
// them can be moved before the wait.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[32]) { tmem_ld_32x32b_x32(taddr, v); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// Arrive on an mbarrier of a CTA of the pair (shared::cluster address).  What the arrival hands over
// are tensor memory reads that have completed (tcgen05.wait::ld), so it needs no release at cluster
// scope, which would wait for every memory access of the thread: 185 -> 111 us at 4096^3.
__device__ __forceinline__ void mbar_arrive_peer(uint32_t cbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cbar) : "memory");
}

// FRAG: 32 rows x 16 columns in pieces of 8 x 2 per four lanes: lane l gets rows l / 4 + 8 i and columns
// 8 n + 2 (l % 4) + {0, 1} in v[8 (i / 2) + 4 n + 2 (i % 2) + {0, 1}].
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {   // lanes 0..15, 16..31
    uint32_t *o = v + 8 * h;
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7])
                 : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16)));
  }
}
template <class Cfg>
__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, uint32_t (&v)[Cfg::CHUNK]) {
  if constexpr (Cfg::FRAG)
    tmem_ld_frag(taddr, v);
  else
    tmem_ld(taddr, v);
}

// A CTA's work: tiles t = first, first + step, ... and the blocks [kb0, kb1) of each.
template <class Cfg>
struct Fp8Work {
  int first, step, kb0, kb1;
  __device__ explicit Fp8Work(const Fp8TcParams &p) {
    if constexpr (Cfg::GROUP == 2) {
      first = cluster_id_x();
      step = cluster_count_x();
      kb0 = 0;
      kb1 = p.kblocks;
    } else {   // one tile per cluster, its blocks shared out over the cluster's CTAs
      first = blockIdx.x / p.split;
      step = p.num_tiles;
      const int r = blockIdx.x % p.split;   // the CTA's rank: clusters are p.split CTAs along x
      kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * r / p.split);
      kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (r + 1) / p.split);
    }
  }
};

// First row of this CTA's 128 rows and first column of the tile.
template <class Cfg>
__device__ __forceinline__ void fp8_tile(const Fp8TcParams &p, int t, uint32_t rank, int &r0, int &c0) {
  int tr, tc;
  tile_coords(t, p.tiles_r, p.tiles_c, p.group, tr, tc);
  r0 = tr * 128 * Cfg::GROUP + (Cfg::GROUP == 2 ? 128 * static_cast<int>(rank) : 0);
  c0 = tc * Cfg::BN;
}

// ------------------------------------------------------------------ producer
template <class Cfg>
__device__ __forceinline__ void fp8_produce(const Fp8TcParams &p, const CUtensorMap *tm_row,
                                            const CUtensorMap *tm_col, uint32_t sbase, const Fp8Bars<Cfg> &bar,
                                            uint32_t rank) {
  const Fp8Work<Cfg> w(p);
  uint32_t it = 0;
  bool ok = true;
  for (int t = w.first; t < p.num_tiles && ok; t += w.step) {
    int r0, c0;
    fp8_tile<Cfg>(p, t, rank, r0, c0);
    if (Cfg::GROUP == 2) c0 += Cfg::BN / 2 * static_cast<int>(rank);
    for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
      const uint32_t s = it % Cfg::STAGES, round = it / Cfg::STAGES;
      if (round > 0 && !wait_parity_bounded(bar.empty(s), (round - 1) & 1, p.wait_budget_ns, p.status)) {
        ok = false;
        break;
      }
      const uint32_t st = sbase + s * Cfg::STAGE_BYTES;
      const int k0 = kb * 128;
      const int rx = p.row_inner ? r0 : k0, ry = p.row_inner ? k0 : r0;
      const int cx = p.col_inner ? (Cfg::HALF_ROWS ? c0 & ~127 : c0) : k0, cy = p.col_inner ? k0 : c0;
      if constexpr (Cfg::GROUP == 2) {
        // both CTAs' copies are counted on the even CTA's barrier
        if (rank == 0) mbar_arrive_expect_tx(bar.full(s), 2 * Cfg::STAGE_BYTES);
        const uint32_t full = map_to_rank(bar.full(s), 0);
        tma_load_2d_pair(st, tm_row, full, rx, ry);
        tma_load_2d_pair(st + Cfg::ROW_BYTES, tm_col, full, cx, cy);
      } else {
        mbar_arrive_expect_tx(bar.full(s), Cfg::HALF_ROWS && !p.col_inner ? Cfg::ROW_BYTES + Cfg::COL_BYTES / 2
                                                                         : Cfg::STAGE_BYTES);
        tma_load_2d(st, tm_row, bar.full(s), rx, ry);
        tma_load_2d(st + Cfg::ROW_BYTES, tm_col, bar.full(s), cx, cy);
      }
    }
  }
  if (rank == 0) {   // the copies in flight land before the CTA may end, whichever role gave up
    for (uint32_t j = it > Cfg::STAGES ? it - Cfg::STAGES : 0; j < it; ++j)
      wait_parity_bounded(bar.full(j % Cfg::STAGES), (j / Cfg::STAGES) & 1, p.wait_budget_ns, nullptr);
  }
}

// ------------------------------------------------------------------ loaders
// 16 bytes from x of row y of a stored matrix, one by one, zeros outside.
__device__ __forceinline__ uint4 load16(const unsigned char *q, int64_t ld, int rows, int cols, int y, int x) {
  uint32_t w[4] = {0, 0, 0, 0};
  if (y < rows) {
    const unsigned char *p = q + y * ld + x;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (x + i < cols) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// One box of 128 rows of 128 bytes at (y0, x0) by 128 threads, in the layout a 128-byte-swizzled TMA box has:
// eight threads a row, sixteen rows at a time.  A thread whose first and last pieces can be read by words reads
// all eight so, twenty loads in flight.
__device__ __forceinline__ void load_box(uint32_t dst, const unsigned char *q, int64_t ld, int rows, int cols, int y0,
                                         int x0, int thread) {
  const int c = thread % 8, r0 = thread / 8, x = x0 + 16 * c;
  const auto put = [&](int r, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 128 * r + 16 * (c ^ (r & 7))), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
  };
  const unsigned char *first = q + (y0 + r0) * ld + x, *last = first + 112 * ld;
  const bool words = y0 + r0 + 112 < rows && x + 16 <= cols &&
                     (reinterpret_cast<uintptr_t>(first) & ~uintptr_t(3)) >= reinterpret_cast<uintptr_t>(q) &&
                     (reinterpret_cast<uintptr_t>(last) & ~uintptr_t(3)) + 20 <=
                         reinterpret_cast<uintptr_t>(q + (rows - 1) * ld + cols);
  if (words) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      uint32_t v[4][5], shift[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(first + 16 * (i + k) * ld);
        const uint32_t *s = reinterpret_cast<const uint32_t *>(at & ~uintptr_t(3));
        shift[k] = 8 * static_cast<uint32_t>(at & 3);
#pragma unroll
        for (int j = 0; j < 5; ++j) v[k][j] = s[j];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        put(r0 + 16 * (i + k), make_uint4(__funnelshift_r(v[k][0], v[k][1], shift[k]), __funnelshift_r(v[k][1], v[k][2], shift[k]),
                                          __funnelshift_r(v[k][2], v[k][3], shift[k]), __funnelshift_r(v[k][3], v[k][4], shift[k])));
    }
  } else {
#pragma unroll 1
    for (int r = r0; r < 128; r += 16) put(r, load16(q, ld, rows, cols, y0 + r, x));
  }
}
template <class Cfg>
__device__ __forceinline__ void fp8_load(const Fp8TcParams &p, uint32_t sbase, const Fp8Bars<Cfg> &bar, int thread) {
  const Fp8Work<Cfg> w(p);
  uint32_t it = 0;
  for (int t = w.first; t < p.num_tiles; t += w.step) {
    int r0, c0;
    fp8_tile<Cfg>(p, t, 0, r0, c0);
    for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
      const uint32_t s = it % Cfg::STAGES, round = it / Cfg::STAGES;
      if (round > 0 && !wait_parity_bounded(bar.empty(s), (round - 1) & 1, p.wait_budget_ns, p.status)) return;
      const uint32_t st = sbase + s * Cfg::STAGE_BYTES;
      const int k0 = kb * 128;
      if (p.row_inner)
        load_box(st, p.row_q, p.row_qld, p.k, p.rows, k0, r0, thread);
      else
        load_box(st, p.row_q, p.row_qld, p.rows, p.k, r0, k0, thread);
      if (p.col_inner)
        load_box(st + Cfg::ROW_BYTES, p.col_q, p.col_qld, p.k, p.cols, k0, c0, thread);
      else
        load_box(st + Cfg::ROW_BYTES, p.col_q, p.col_qld, p.cols, p.k, c0, k0, thread);
      fence_proxy_async_smem();   // the tensor cores read through the async proxy
      mbar_arrive(bar.full(s));
    }
  }
}

// ------------------------------------------------------------------ MMA issue
template <class Cfg>
__device__ __forceinline__ void fp8_issue(const Fp8TcParams &p, uint32_t sbase, uint32_t tmem,
                                          const Fp8Bars<Cfg> &bar) {
  const Fp8Work<Cfg> w(p);
  const uint32_t row_step = p.row_inner ? 4096 : 32, col_step = p.col_inner ? 4096 : 32;
  uint32_t it = 0;
  bool ok = true;
  for (int t = w.first; t < p.num_tiles && ok; t += w.step) {
    uint32_t col_off = Cfg::ROW_BYTES;   // of the tile's columns in a stage
    if (Cfg::HALF_ROWS && p.col_inner) {
      int r0, c0;
      fp8_tile<Cfg>(p, t, 0, r0, c0);
      col_off += c0 & 64;
    }
    for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
      const uint32_t b = it % Cfg::ACCS, use = it / Cfg::ACCS;
      const uint32_t s = it % Cfg::STAGES, round = it / Cfg::STAGES;
      // the copies are usually there first: the accumulator's hand-over is the shorter way to the MMA
      ok = wait_parity_bounded(bar.full(s), round & 1, p.wait_budget_ns, p.status) &&
           (use == 0 || wait_parity_bounded(bar.acc_empty(b), (use - 1) & 1, p.wait_budget_ns, p.status));
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t st = sbase + s * Cfg::STAGE_BYTES, d = tmem + b * Cfg::BN;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_fp8<Cfg::GROUP>(d, desc_fp8(st + kk * row_step), desc_fp8(st + col_off + kk * col_step), p.idesc,
                            kk > 0);
      if constexpr (Cfg::GROUP == 2) {
        mma_commit_pair(bar.empty(s), 0x3);
        mma_commit_pair(bar.acc_full(b), 0x3);
      } else {
        mma_commit(bar.empty(s));
        mma_commit(bar.acc_full(b));
      }
    }
  }
  // every MMA issued is complete before tensor memory is released
  if constexpr (Cfg::GROUP == 2)
    mma_commit_pair(bar.drain(), 0x1);
  else
    mma_commit(bar.drain());
  wait_parity_bounded(bar.drain(), 0, p.wait_budget_ns, nullptr);
}

// ------------------------------------------------------------------ scales
// Index of the scale of outer index o and block kb.
__device__ __forceinline__ int64_t scale_index(int o, int kb, int shift, int inner, int64_t ld) {
  const int64_t i = o >> shift;
  return inner ? kb * ld + i : i * ld + kb;
}

// 16-byte asynchronous copy global -> shared; src_bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// One warp: the scales of SCALE_BLOCKS blocks of a tile into slot g % SLOTS.
template <class Cfg>
__device__ __forceinline__ void fp8_scales(const Fp8TcParams &p, uint32_t sbase, const Fp8Bars<Cfg> &bar,
                                           uint32_t rank, int lane) {
  constexpr int SB = Cfg::SCALE_BLOCKS;
  const Fp8Work<Cfg> w(p);
  uint32_t g = 0;
  bool ok = true;
  for (int t = w.first; t < p.num_tiles && ok; t += w.step) {
    int r0, c0;
    fp8_tile<Cfg>(p, t, rank, r0, c0);
    for (int kb0 = w.kb0; kb0 < w.kb1; kb0 += SB, ++g) {
      const uint32_t slot = g % Cfg::SCALE_SLOTS, round = g / Cfg::SCALE_SLOTS;
      if (round > 0 && !wait_parity_bounded(bar.sc_empty(slot), (round - 1) & 1, p.wait_budget_ns, p.status)) {
        ok = false;
        break;
      }
      const uint32_t dst = sbase + Cfg::SCALE_OFFSET + slot * Cfg::SCALE_BYTES;
      const int n = min(SB, w.kb1 - kb0);
      const bool vec = p.row_vec && kb0 % SB == 0 && kb0 + SB <= p.kblocks;
#pragma unroll 1
      for (int i = lane; i < 128; i += 32) {
        const bool in = r0 + i < p.rows;
        const float *src = p.row_s + scale_index(in ? r0 + i : 0, kb0, p.row_shift, p.row_inner, p.row_ld);
        if (vec) {
          cp_async_16(dst + 16 * i, src, in ? 16 : 0);
        } else {
          const int64_t step = p.row_inner ? p.row_ld : 1;
          for (int k = 0; k < n; ++k, src += step) cp_async_4(dst + 16 * i + 4 * k, src, in ? 4 : 0);
        }
      }
#pragma unroll 1
      for (int i = lane; i < Cfg::BN; i += 32) {
        const int c = c0 + i;
        const bool in = c < p.cols;
        const float *src = p.col_s + scale_index(in ? c : 0, kb0, p.col_shift, p.col_inner, p.col_ld);
        const int64_t step = p.col_inner ? p.col_ld : 1;
        for (int k = 0; k < n; ++k, src += step)
          cp_async_4(dst + 4 * (Cfg::COL_SCALES + k * Cfg::BN + i), src, in ? 4 : 0);
      }
      cp_async_mbar_arrive_noinc(bar.sc_full(slot));
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ output
// n <= 8 consecutive elements of a row of C.
template <class T>
__device__ __forceinline__ void fp8_put8(const Fp8TcParams &p, T *c, const float (&v)[8], int n) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = p.alpha * v[i];
  if (p.beta != 0.0f) {
    float old[8];
    unpack(load8(c, n, p.vecC), old);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] += p.beta * old[i];
  }
  store8(c, o, n, p.vecC);
}
template <class T>
__device__ __forceinline__ void fp8_put1(const Fp8TcParams &p, T *c, float v) {
  v *= p.alpha;
  if (p.beta != 0.0f) v += p.beta * to_float(*c);
  from_float(c, v);
}
// FRAG: row and column, in the warp's 32 x ECOLS, of a thread's sums j and j + 1 (j even).
template <class Cfg>
__device__ __forceinline__ int frag_row(int j, int lane) {
  return lane / 4 + 16 * (j % Cfg::CHUNK / (Cfg::CHUNK / 2)) + 8 * (j / 2 % 2);
}
template <class Cfg>
__device__ __forceinline__ int frag_col(int j, int lane) {
  return j / Cfg::CHUNK * Cfg::CHUNK + j % (Cfg::CHUNK / 2) / 4 * 8 + 2 * (lane & 3);
}

// Two consecutive elements of a row of C at an even column, the second if `two`.
template <class T>
__device__ __forceinline__ void fp8_put2(const Fp8TcParams &p, T *c, float v0, float v1, bool two) {
  if (!two || !p.vecC) {
    fp8_put1(p, c, v0);
    if (two) fp8_put1(p, c + 1, v1);
    return;
  }
  v0 *= p.alpha;
  v1 *= p.alpha;
  if (p.beta != 0.0f) {
    v0 += p.beta * to_float(c[0]);
    v1 += p.beta * to_float(c[1]);
  }
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float2 *>(c) = make_float2(v0, v1);
  else
    *reinterpret_cast<uint32_t *>(c) = pack2(v0, v1, T());
}
// The first n (of four, or more) consecutive elements of a row of C, at a multiple of four.
template <class T>
__device__ __forceinline__ void fp8_put4(const Fp8TcParams &p, T *c, float4 v, int n) {
  float o[4] = {p.alpha * v.x, p.alpha * v.y, p.alpha * v.z, p.alpha * v.w};
  if (p.beta != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) o[i] += p.beta * to_float(c[i]);
  }
  if (n >= 4 && p.vecC) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4 *>(c) = make_float4(o[0], o[1], o[2], o[3]);
    else
      *reinterpret_cast<uint2 *>(c) = make_uint2(pack2(o[0], o[1], T()), pack2(o[2], o[3], T()));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) from_float(c + i, o[i]);
  }
}
// The sums of a warp's 32 rows from r and ECOLS columns from c0: a thread holds those of row r + lane, or
// (FRAG) pieces of four rows.  `stage`: the warp's STORE_BYTES of shared memory (STAGED).
template <class Cfg, class T>
__device__ __forceinline__ void fp8_store(const Fp8TcParams &p, int r, int c0, int lane, uint32_t stage,
                                          const float (&acc)[Cfg::ECOLS]) {
  T *C = static_cast<T *>(p.C);
  if constexpr (Cfg::FRAG) {
#pragma unroll
    for (int j = 0; j < Cfg::ECOLS; j += 2) {
      const int row = r + frag_row<Cfg>(j, lane), col = c0 + frag_col<Cfg>(j, lane);
      if (row < p.rows && col < p.cols) fp8_put2(p, C + row * p.ldc + col, acc[j], acc[j + 1], col + 1 < p.cols);
    }
  } else if constexpr (Cfg::SWAP) {
    if (r + lane < p.rows) {
#pragma unroll
      for (int j = 0; j < Cfg::ECOLS; ++j)
        if (c0 + j < p.cols) fp8_put1(p, C + (c0 + j) * p.ldc + r + lane, acc[j]);
    }
  } else if (!Cfg::STAGED || p.vecC) {
    if (r + lane < p.rows) {
#pragma unroll
      for (int j = 0; j < Cfg::ECOLS; j += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = acc[j + i];
        const int n = p.cols - (c0 + j);
        if (n > 0) fp8_put8(p, C + (r + lane) * p.ldc + c0 + j, v, n < 8 ? n : 8);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < Cfg::ECOLS; j += 16) {
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        sts128(stage + 4 * (lane * Cfg::STORE_PITCH + i),
               make_float4(acc[j + i], acc[j + i + 1], acc[j + i + 2], acc[j + i + 3]));
      __syncwarp();
      const int at = lane & 15, c = c0 + j + at;   // two rows at a time
      if (c < p.cols) {
#pragma unroll 1
        for (int row = lane >> 4; row < 32; row += 16) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(v[i])
                         : "r"(stage + 4 * ((row + 2 * i) * Cfg::STORE_PITCH + at)));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (r + row + 2 * i < p.rows) fp8_put1(p, C + (r + row + 2 * i) * p.ldc + c, v[i]);
        }
      }
      __syncwarp();
    }
  }
}

// BULK: the same through shared memory and TMA stores (columns and rows past the edge are not written).  The
// warp's last stores have read the place before it is written again.
template <class Cfg, class T>
__device__ __forceinline__ void fp8_store_bulk(const Fp8TcParams &p, const CUtensorMap *tm_c, int r, int c0, int lane,
                                               uint32_t stage, const float (&acc)[Cfg::ECOLS]) {
  constexpr int BOX = 128 / sizeof(T), COLS = Cfg::STORE_BYTES / 32 / sizeof(T);   // columns of a box, of a pass
  // column `col` of the pass and row `row`: boxes of 32 rows, 16-byte units exchanged as the map's swizzle does
  const auto place = [&](int row, int col) {
    const int unit = col % BOX * static_cast<int>(sizeof(T)) / 16, rest = col * static_cast<int>(sizeof(T)) % 16;
    return stage + col / BOX * 4096 + 128 * row + 16 * (unit ^ (row & 7)) + rest;
  };
#pragma unroll
  for (int j0 = 0; j0 < Cfg::ECOLS; j0 += COLS) {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
    if constexpr (Cfg::FRAG) {
#pragma unroll
      for (int j = 0; j < COLS; j += 2) {
        const uint32_t to = place(frag_row<Cfg>(j0 + j, lane), frag_col<Cfg>(j0 + j, lane) - j0);
        const float v0 = p.alpha * acc[j0 + j], v1 = p.alpha * acc[j0 + j + 1];
        if constexpr (sizeof(T) == 4)
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v0), "f"(v1) : "memory");
        else
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(pack2(v0, v1, T())) : "memory");
      }
    } else {
#pragma unroll
      for (int j = 0; j < COLS; j += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p.alpha * acc[j0 + j + i];
        Raw<T> o;
        pack(o, v);
#pragma unroll
        for (int u = 0; u < static_cast<int>(sizeof(o) / 16); ++u)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(place(lane, j + 4 * u)), "r"(o.u[u].x),
                       "r"(o.u[u].y), "r"(o.u[u].z), "r"(o.u[u].w)
                       : "memory");
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && r < p.rows) {
#pragma unroll
      for (int j = 0; j < COLS; j += BOX)
        if (c0 + j0 + j < p.cols) tma_store_2d(tm_c, stage + j / BOX * 4096, c0 + j0 + j, r);
      bulk_commit_group();
    }
  }
}

// The cluster barrier's halves.  Threads that have read what they want from the other CTAs arrive (release:
// their reads come before it), and the last wait keeps every CTA's shared memory alive until all have.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// This CTA's share (rows rank * 128 / SPLIT ..) of a tile whose partial sums lie in the shared memory of
// the cluster's CTAs: they are added in the CTAs' order, four elements of a row of C at a time.  All of a
// thread's reads are in flight at once, and the CTA is done with its peers before it writes C.
template <class Cfg, int SPLIT>
__device__ __forceinline__ void fp8_reduce(const Fp8TcParams &p, uint32_t sbase, uint32_t rank, int r0, int c0) {
  constexpr int ROWS = 128 / SPLIT, LINE = Cfg::SWAP ? ROWS : Cfg::BN;   // elements of a line that are this CTA's
  constexpr int UNITS = ROWS * Cfg::BN / 4, THREADS = 32 * Cfg::EPI_WARPS, PER = (UNITS + THREADS - 1) / THREADS;
  const int first = ROWS * static_cast<int>(rank);
  const auto line_of = [&](int u) { return u / (LINE / 4) + (Cfg::SWAP ? 0 : first); };
  const auto at_of = [&](int u) { return u % (LINE / 4) * 4 + (Cfg::SWAP ? first : 0); };
  float4 x[PER][SPLIT];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int u = min(static_cast<int>(threadIdx.x) - 128 + k * THREADS, UNITS - 1);
    const uint32_t at = sbase + 4 * (line_of(u) * Cfg::PART_PITCH + at_of(u));
#pragma unroll
    for (int i = 0; i < SPLIT; ++i) x[k][i] = ld_dsmem_v4(map_to_rank(at, i));
  }
#pragma unroll
  for (int k = 0; k < PER; ++k)
#pragma unroll
    for (int i = 1; i < SPLIT; ++i) {
      x[k][0].x += x[k][i].x;
      x[k][0].y += x[k][i].y;
      x[k][0].z += x[k][i].z;
      x[k][0].w += x[k][i].w;
    }
  __syncwarp();
  cluster_arrive();
  const int line0 = Cfg::SWAP ? c0 : r0, at0 = Cfg::SWAP ? r0 : c0;
  const int lines = Cfg::SWAP ? p.cols : p.rows, length = Cfg::SWAP ? p.rows : p.cols;
  const auto store = [&](auto type) {
    using T = decltype(type);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int u = threadIdx.x - 128 + k * THREADS;
      const int line = line0 + line_of(u), at = at0 + at_of(u);
      if (u < UNITS && line < lines && at < length)
        fp8_put4(p, static_cast<T *>(p.C) + line * p.ldc + at, x[k][0], length - at);
    }
  };
  if (p.typeC == SGEMM_TYPE_F32)
    store(float());
  else if (p.typeC == SGEMM_TYPE_BF16)
    store(__nv_bfloat16());
  else
    store(__half());
}

// ------------------------------------------------------------------ epilogue
// The loads of tensor memory run one chunk ahead of the sums, across blocks too: before the last chunk of a
// block is added, its accumulator has been handed back and the next block's first chunk is on its way.  (FRAG:
// a chunk's scales are multiplied while its own load is on its way, which takes as long; 381 -> 363 us at
// 4096 x 4096 x 16384.)
template <class Cfg>
__device__ __forceinline__ void fp8_epilogue(const Fp8TcParams &p, unsigned char *smem, uint32_t sbase, uint32_t tmem,
                                             const Fp8Bars<Cfg> &bar, uint32_t rank, int q, int half, int lane,
                                             const CUtensorMap *tm_c) {
  constexpr int EC = Cfg::ECOLS, CH = Cfg::CHUNK, NC = EC / CH, SB = Cfg::SCALE_BLOCKS;
  const Fp8Work<Cfg> w(p);
  const uint32_t src = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * EC;
  const int row = 32 * q + lane;
  uint32_t it = 0, group = 0;   // blocks and slots of scales used so far
  // accumulator of block `i` is complete (whole warps: the loads want them)
  const auto acc_ready = [&](uint32_t i) {
    const bool ok = wait_parity_bounded(bar.acc_full(i % Cfg::ACCS), i / Cfg::ACCS & 1, p.wait_budget_ns, p.status);
    if (!__all_sync(~0u, ok)) return false;
    tc_fence_after_sync();
    return true;
  };
  for (int t = w.first; t < p.num_tiles; t += w.step) {
    int r0, c0;
    fp8_tile<Cfg>(p, t, rank, r0, c0);
    float acc[EC];
#pragma unroll
    for (int j = 0; j < EC; ++j) acc[j] = 0.0f;
    uint32_t v[2][CH];
    // !VEC: one scale per thread and block, loaded a block ahead (in groups of four, 16 bytes at a time,
    // it was slower: 245 -> 258 us at 4096 x 4096 x 16384).  Those of a row past the edge are the last
    // one's: its sums are not stored.
    const float *rp = p.row_s + scale_index(min(r0 + row, p.rows - 1), w.kb0, p.row_shift, p.row_inner, p.row_ld);
    const float *cp = p.col_s + scale_index(min(c0 + half * EC, p.cols - 1), w.kb0, p.col_shift, p.col_inner, p.col_ld);
    const int64_t rstep = p.row_inner ? p.row_ld : 1, cstep = p.col_inner ? p.col_ld : 1;
    float row_s = 0.0f, col_s = 0.0f;
    if (!Cfg::VEC && w.kb0 < w.kb1) {
      row_s = *rp;
      col_s = *cp;
    }
    if (w.kb0 < w.kb1) {
      if (!acc_ready(it)) return;
      if (!Cfg::FRAG) tmem_ld_chunk<Cfg>(src + it % Cfg::ACCS * Cfg::BN, v[0]);
    }
    const float *sc = reinterpret_cast<const float *>(smem + Cfg::SCALE_OFFSET);   // VEC: the slot's scales
    for (int kb = w.kb0, i = 0; kb < w.kb1; ++kb, ++it) {   // i: block of its slot of scales
      const uint32_t b = it % Cfg::ACCS;
      const bool more = kb + 1 < w.kb1;
      float2 rs[4];   // FRAG: the scales of the thread's four rows; else of its one
      if constexpr (Cfg::VEC) {
        if (i == 0) {
          const uint32_t slot = group % Cfg::SCALE_SLOTS;
          const bool ok = wait_parity_bounded(bar.sc_full(slot), group / Cfg::SCALE_SLOTS & 1, p.wait_budget_ns, p.status);
          if (!__all_sync(~0u, ok)) return;
          sc = reinterpret_cast<const float *>(smem + Cfg::SCALE_OFFSET + slot * Cfg::SCALE_BYTES);
        }
#pragma unroll
        for (int j = 0; j < (Cfg::FRAG ? 4 : 1); ++j) {
          const float f = sc[(Cfg::FRAG ? 32 * q + lane / 4 + 8 * j : row) * SB + i];
          rs[j] = make_float2(f, f);
        }
      } else {
        const float f = row_s * col_s;
        rs[0] = make_float2(f, f);
        if (more) {
          row_s = *(rp += rstep);
          col_s = *(cp += cstep);
        }
      }
      const float *cols = sc + Cfg::COL_SCALES + i * Cfg::BN + half * EC;
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) {
        uint32_t(&x)[CH] = v[Cfg::FRAG ? 0 : cc & 1];
        if constexpr (Cfg::FRAG) tmem_ld_chunk<Cfg>(src + b * Cfg::BN + cc * CH, x);
        // the columns' scales, before the values are there: of the chunk's columns, or (FRAG) of the
        // thread's pairs of them, times its rows'
        float2 f[CH / 2];
        if constexpr (Cfg::FRAG) {
          float2 u[CH / 8];
#pragma unroll
          for (int n = 0; n < CH / 8; ++n) u[n] = *reinterpret_cast<const float2 *>(cols + cc * CH + 8 * n + 2 * (lane & 3));
#pragma unroll
          for (int j = 0; j < CH; j += 2) f[j / 2] = __fmul2_rn(u[j % (CH / 2) / 4], rs[j / (CH / 2) * 2 + j / 2 % 2]);
        } else if constexpr (Cfg::VEC) {
#pragma unroll
          for (int j = 0; j < CH; j += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(cols + cc * CH + j);
            f[j / 2] = __fmul2_rn(make_float2(u.x, u.y), rs[0]);
            f[j / 2 + 1] = __fmul2_rn(make_float2(u.z, u.w), rs[0]);
          }
        }
        tmem_ld_wait_for(x);
        if (cc + 1 < NC) {
          if (!Cfg::FRAG) tmem_ld_chunk<Cfg>(src + b * Cfg::BN + (cc + 1) * CH, v[(cc + 1) & 1]);
        } else {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (Cfg::GROUP == 2 && rank != 0)
              mbar_arrive_peer(map_to_rank(bar.acc_empty(b), 0));
            else
              mbar_arrive(bar.acc_empty(b));
          }
          if (more) {
            if (!acc_ready(it + 1)) return;
            if (!Cfg::FRAG) tmem_ld_chunk<Cfg>(src + (it + 1) % Cfg::ACCS * Cfg::BN, v[0]);
          }
        }
#pragma unroll
        for (int j = 0; j < CH; j += 2) {
          float *o = acc + cc * CH + j;
          const float2 a = make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
          const float2 c = Cfg::VEC ? f[j / 2] : rs[0];
          const float2 sum = __ffma2_rn(a, c, make_float2(o[0], o[1]));
          o[0] = sum.x;
          o[1] = sum.y;
        }
      }
      if constexpr (Cfg::VEC) {
        if (++i == SB || !more) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar.sc_empty(group % Cfg::SCALE_SLOTS));
          ++group;
          i = 0;
        }
      }
    }
    if (Cfg::GROUP == 1 && p.split > 1) {
      // every MMA of this CTA has completed, so the stage ring is free
      if constexpr (Cfg::FRAG) {
#pragma unroll
        for (int j = 0; j < EC; j += 2) {
          const int r = 32 * q + frag_row<Cfg>(j, lane), c = half * EC + frag_col<Cfg>(j, lane);
          *reinterpret_cast<float2 *>(smem + 4 * (r * Cfg::PART_PITCH + c)) = make_float2(acc[j], acc[j + 1]);
        }
      } else if constexpr (Cfg::SWAP) {
#pragma unroll
        for (int j = 0; j < EC; ++j) reinterpret_cast<float *>(smem)[j * Cfg::PART_PITCH + row] = acc[j];
      } else {
#pragma unroll
        for (int j = 0; j < EC; j += 4)
          sts128(sbase + 4 * (row * Cfg::PART_PITCH + half * EC + j),
                 make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
      }
    } else {
      const int c = c0 + half * EC, r = r0 + 32 * q;
      const uint32_t stage = sbase + Cfg::STORE_OFFSET + (q + 4 * half) * Cfg::STORE_BYTES;
      if constexpr (Cfg::BULK) {
        if (p.typeC == SGEMM_TYPE_F32)
          fp8_store_bulk<Cfg, float>(p, tm_c, r, c, lane, stage, acc);
        else if (p.typeC == SGEMM_TYPE_BF16)
          fp8_store_bulk<Cfg, __nv_bfloat16>(p, tm_c, r, c, lane, stage, acc);
        else
          fp8_store_bulk<Cfg, __half>(p, tm_c, r, c, lane, stage, acc);
      } else if (p.typeC == SGEMM_TYPE_F32)
        fp8_store<Cfg, float>(p, r, c, lane, stage, acc);
      else if (p.typeC == SGEMM_TYPE_BF16)
        fp8_store<Cfg, __nv_bfloat16>(p, r, c, lane, stage, acc);
      else
        fp8_store<Cfg, __half>(p, r, c, lane, stage, acc);
    }
  }
}

// ------------------------------------------------------------------ kernel
template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, Cfg::CTAS)
    fp8_tc_kernel(const __grid_constant__ CUtensorMap tm_row, const __grid_constant__ CUtensorMap tm_col,
                  const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ Fp8TcParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                          ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const Fp8Bars<Cfg> bar{sbase + Cfg::BAR_OFFSET};
  const uint32_t slot = sbase + Cfg::BAR_OFFSET + Cfg::NUM_BARS * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool shared_tile = Cfg::GROUP == 1 && p.split > 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(bar.full(s), Cfg::LOAD ? 128 : 1);
      mbar_init(bar.empty(s), 1);
    }
    for (int b = 0; b < Cfg::ACCS; ++b) {
      mbar_init(bar.acc_full(b), 1);
      mbar_init(bar.acc_empty(b), Cfg::GROUP * Cfg::EPI_WARPS);
    }
    for (int r = 0; r < Cfg::SCALE_SLOTS; ++r) {
      mbar_init(bar.sc_full(r), 32);
      mbar_init(bar.sc_empty(r), Cfg::EPI_WARPS);
    }
    mbar_init(bar.drain(), 1);
    fence_mbar_init();
    if (!Cfg::LOAD) {
      tma_prefetch_desc(&tm_row);
      tma_prefetch_desc(&tm_col);
      if (Cfg::BULK) tma_prefetch_desc(&tm_c);
    }
  }
  if (warp == 1) {
    if constexpr (Cfg::GROUP == 2)
      tmem_alloc_pair(slot, Cfg::TMEM_COLS);
    else
      tmem_alloc(slot, Cfg::TMEM_COLS);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (Cfg::GROUP == 2) cluster_sync();   // the peer's copies and arrivals need initialised barriers
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + Cfg::BAR_OFFSET + Cfg::NUM_BARS * 8);
  griddep_wait();
  griddep_launch_dependents();   // this CTA has its tensor memory: a dependent cannot take it first

  if (warp < 4) {
    if constexpr (Cfg::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_WG0));
    if (warp == 0) {
      if (!Cfg::LOAD && lane == 0) fp8_produce<Cfg>(p, &tm_row, &tm_col, sbase, bar, Cfg::GROUP == 2 ? rank : 0);
    } else if (warp == 1) {
      if (lane == 0 && (Cfg::GROUP == 1 || rank == 0)) fp8_issue<Cfg>(p, sbase, tmem, bar);
    } else if (Cfg::VEC && warp == 2) {
      fp8_scales<Cfg>(p, sbase, bar, rank, lane);
    }
    __syncwarp();
    if (shared_tile) {
      cluster_sync();
      cluster_arrive();
    }
  } else if (Cfg::LOAD && warp >= 4 + Cfg::EPI_WARPS) {
    fp8_load<Cfg>(p, sbase, bar, threadIdx.x - 128 - 32 * Cfg::EPI_WARPS);
    __syncwarp();
    if (shared_tile) {
      cluster_sync();
      cluster_arrive();
    }
  } else {
    if constexpr (Cfg::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::REGS_EPI));
    fp8_epilogue<Cfg>(p, smem, sbase, tmem, bar, rank, warp & 3, (warp >> 2) - 1, lane, &tm_c);
    // whatever ended the epilogue: its stores are done with this CTA's shared memory, and its loads with the
    // tensor memory, before those may go
    if (Cfg::BULK && lane == 0) bulk_wait_group_all();
    __syncwarp();
    tmem_ld_wait();
    if (shared_tile) {
      cluster_sync();   // every CTA's partial tile is written
      int r0, c0;
      fp8_tile<Cfg>(p, blockIdx.x / p.split, 0, r0, c0);
      if (p.split == 2)
        fp8_reduce<Cfg, 2>(p, sbase, rank, r0, c0);
      else if (p.split == 4)
        fp8_reduce<Cfg, 4>(p, sbase, rank, r0, c0);
      else
        fp8_reduce<Cfg, 8>(p, sbase, rank, r0, c0);
      __syncwarp();
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (Cfg::GROUP == 2) cluster_sync();   // no CTA of a pair releases tensor memory early
  if (shared_tile) cluster_wait();
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (Cfg::GROUP == 2)
      tmem_dealloc_pair(tmem, Cfg::TMEM_COLS);
    else
      tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

}  // namespace sg
