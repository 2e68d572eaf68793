// fp8_checks.h -- argument checks of the 8-bit layer's C ABI (host side),
// shared by its entry points.
#pragma once

#include "dispatch.h"
#include "sgemm_fp8.h"

namespace sg {

inline bool is_float_type(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_BF16 || t == SGEMM_TYPE_F16; }
inline bool is_fp8_type(int t) { return t == SGEMM_TYPE_E4M3 || t == SGEMM_TYPE_E5M2; }
inline int type_size(int t) { return t == SGEMM_TYPE_F32 ? 4 : is_fp8_type(t) ? 1 : 2; }

inline bool good_dim(int64_t v) { return v >= 0 && v <= kMaxDim; }
inline bool good_ld(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1) && ld <= kMaxLd; }
inline int64_t blocks_of(int64_t n, int block) { return (n + block - 1) / block; }

// A matrix that a call reads or writes.
struct Range {
  const void *p;
  int64_t rows, cols, ld;
  int elem;
  bool output;
};

// Present, inside the address space, elements on their own alignment, outputs
// apart from everything else.  A range of null pointer and no rows stands for
// an argument that was not given.
template <int N>
sgemm_status_t check_ranges(const Range (&r)[N]) {
  using u128 = unsigned __int128;
  u128 lo[N], hi[N];
  for (int i = 0; i < N; ++i) {
    lo[i] = hi[i] = 0;
    if (r[i].rows == 0 || r[i].cols == 0) continue;
    if (!r[i].p) return SGEMM_ERR_INVALID_VALUE;
    lo[i] = reinterpret_cast<uintptr_t>(r[i].p);
    if (lo[i] % r[i].elem != 0) return SGEMM_ERR_INVALID_VALUE;
    hi[i] = lo[i] + static_cast<u128>(r[i].elem) *
                        (static_cast<u128>(r[i].rows - 1) * static_cast<u128>(r[i].ld) + static_cast<u128>(r[i].cols));
    if (hi[i] > static_cast<u128>(1) << 64) return SGEMM_ERR_INVALID_VALUE;
  }
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < N; ++j)
      if (i != j && r[i].output && lo[i] < hi[j] && lo[j] < hi[i]) return SGEMM_ERR_ALIASING;
  return SGEMM_SUCCESS;
}

// The status of a call whose launches returned e.
inline sgemm_status_t queued(cudaError_t e, int launches) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  t_last_launches = launches;
  return SGEMM_SUCCESS;
}

}  // namespace sg
