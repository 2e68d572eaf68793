// fp8_api.cu -- the C ABI of include/sgemm_fp8.h: argument checks (all on the
// host, before anything is queued), the degenerate cases and the dispatch.
#include "sgemm_fp8.h"

#include "dispatch.h"
#include "fp8.h"

namespace sg {
namespace {

using u128 = unsigned __int128;

bool is_float_type(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_BF16 || t == SGEMM_TYPE_F16; }
bool is_fp8_type(int t) { return t == SGEMM_TYPE_E4M3 || t == SGEMM_TYPE_E5M2; }
int type_size(int t) { return t == SGEMM_TYPE_F32 ? 4 : is_fp8_type(t) ? 1 : 2; }

bool good_dim(int64_t v) { return v >= 0 && v <= kMaxDim; }
bool good_ld(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1) && ld <= kMaxLd; }

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
sgemm_status_t check_ranges(const Range *r, int n) {
  u128 lo[12], hi[12];
  for (int i = 0; i < n; ++i) {
    lo[i] = hi[i] = 0;
    if (r[i].rows == 0 || r[i].cols == 0) continue;
    if (!r[i].p) return SGEMM_ERR_INVALID_VALUE;
    lo[i] = reinterpret_cast<uintptr_t>(r[i].p);
    if (lo[i] % r[i].elem != 0) return SGEMM_ERR_INVALID_VALUE;
    hi[i] = lo[i] + static_cast<u128>(r[i].elem) *
                        (static_cast<u128>(r[i].rows - 1) * static_cast<u128>(r[i].ld) + static_cast<u128>(r[i].cols));
    if (hi[i] > static_cast<u128>(1) << 64) return SGEMM_ERR_INVALID_VALUE;
  }
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      if (i != j && r[i].output && lo[i] < hi[j] && lo[j] < hi[i]) return SGEMM_ERR_ALIASING;
  return SGEMM_SUCCESS;
}

sgemm_status_t queued(cudaError_t e, int launches) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SGEMM_ERR_LAUNCH;
  }
  t_last_launches = launches;
  return SGEMM_SUCCESS;
}

int64_t blocks_of(int64_t n, int block) { return (n + block - 1) / block; }

sgemm_status_t quantize(const QuantizeParams &p, int br, int bc, bool both, cudaStream_t stream) {
  const int e = type_size(p.typeX);
  const Range r[5] = {
      {p.x, p.rows, p.cols, p.ldx, e, false},
      {p.qr, both || p.qr ? p.rows : 0, p.cols, p.ldqr, 1, true},
      {p.sr, both || p.qr ? blocks_of(p.rows, both ? 1 : br) : 0, blocks_of(p.cols, both ? 128 : bc), p.ldsr, 4, true},
      {p.qc, both || p.qc ? p.rows : 0, p.cols, p.ldqc, 1, true},
      {p.sc, both || p.qc ? blocks_of(p.rows, 128) : 0, p.cols, p.ldsc, 4, true}};
  const sgemm_status_t st = check_ranges(r, 5);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  if (!device_state(&why)) return why;
  return queued(launch_quantize(p, stream), 1);
}

}  // namespace
}  // namespace sg

using namespace sg;

extern "C" {

sgemm_status_t sgemm_fp8(int transA, int transB, int64_t M, int64_t N, int64_t K, float alpha, const void *A,
                         sgemm_type_t typeA, int64_t lda, const float *SA, int64_t ldsa, int blockA, const void *B,
                         sgemm_type_t typeB, int64_t ldb, const float *SB, int64_t ldsb, int blockB, float beta,
                         void *C, sgemm_type_t typeC, int64_t ldc, void *stream) {
  const int ta = norm_op(transA), tb = norm_op(transB);
  if (ta < 0 || tb < 0 || !good_dim(M) || !good_dim(N) || !good_dim(K)) return SGEMM_ERR_INVALID_VALUE;
  if (!is_fp8_type(typeA) || !is_fp8_type(typeB) || !is_float_type(typeC)) return SGEMM_ERR_INVALID_VALUE;
  if ((blockA != 1 && blockA != 128) || (blockB != 1 && blockB != 128)) return SGEMM_ERR_INVALID_VALUE;
  const int64_t kb = blocks_of(K, SGEMM_FP8_BLOCK), ma = blocks_of(M, blockA), nb = blocks_of(N, blockB);
  if (!good_ld(lda, ta ? M : K) || !good_ld(ldb, tb ? K : N) || !good_ld(ldc, N) || !good_ld(ldsa, ta ? ma : kb) ||
      !good_ld(ldsb, tb ? kb : nb))
    return SGEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) {
    t_last_launches = 0;
    return SGEMM_SUCCESS;
  }
  const bool product = K > 0 && alpha != 0.0f;
  const int64_t has = product ? 1 : 0;
  const Range r[5] = {{C, M, N, ldc, type_size(typeC), true},
                      {A, has * (ta ? K : M), ta ? M : K, lda, 1, false},
                      {SA, has * (ta ? kb : ma), ta ? ma : kb, ldsa, 4, false},
                      {B, has * (tb ? N : K), tb ? K : N, ldb, 1, false},
                      {SB, has * (tb ? nb : kb), tb ? kb : nb, ldsb, 4, false}};
  const sgemm_status_t st = check_ranges(r, 5);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  DeviceState *d = device_state(&why);
  if (!d) return why;
  Fp8Params p;
  p.a = {static_cast<const unsigned char *>(A), SA, lda, ldsa, typeA == SGEMM_TYPE_E5M2, ta == 1, blockA == 128 ? 7 : 0};
  p.b = {static_cast<const unsigned char *>(B), SB, ldb, ldsb, typeB == SGEMM_TYPE_E5M2, tb == 0, blockB == 128 ? 7 : 0};
  p.C = C;
  p.ldc = ldc;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.typeC = typeC;
  p.alpha = alpha;
  p.beta = beta;
  p.wait_budget_ns = g_wait_budget_ns.load(std::memory_order_relaxed);
  p.status = d->status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!product) return queued(launch_fp8_scale_c(p, s), 1);
  return queued(launch_fp8_product(p, d->sm_count, s), 1);
}

int sgemm_fp8_select_form(int transA, int transB, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                          const void *B, int64_t ldb, int blockB, float beta, const void *C, sgemm_type_t typeC,
                          int64_t ldc, int *split) {
  const int ta = norm_op(transA), tb = norm_op(transB);
  if (ta < 0 || tb < 0 || !good_dim(M) || !good_dim(N) || !good_dim(K) || M == 0 || N == 0 || K == 0) return -1;
  if (!is_float_type(typeC) || (blockB != 1 && blockB != 128)) return -1;
  if (!good_ld(lda, ta ? M : K) || !good_ld(ldb, tb ? K : N) || !good_ld(ldc, N)) return -1;
  Fp8Params p = {};
  p.a = {static_cast<const unsigned char *>(A), nullptr, lda, 0, 0, ta == 1, 0};
  p.b = {static_cast<const unsigned char *>(B), nullptr, ldb, 0, 0, tb == 0, blockB == 128 ? 7 : 0};
  p.C = const_cast<void *>(C);
  p.ldc = ldc;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.typeC = typeC;
  p.beta = beta;
  sgemm_status_t why = SGEMM_SUCCESS;
  const DeviceState *d = device_state(&why);
  const Fp8Choice c = choose_fp8_form(p, d ? d->sm_count : 152);
  if (split) *split = c.split;
  return c.form;
}

sgemm_status_t sgemm_fp8_quantize(int64_t rows, int64_t cols, const void *X, sgemm_type_t typeX, int64_t ldx, void *Q,
                                  sgemm_type_t typeQ, int64_t ldq, float *S, int64_t lds, int block_rows,
                                  int block_cols, void *stream) {
  const bool row = block_rows == 1 && block_cols == 128, col = block_rows == 128 && block_cols == 1;
  const bool tile = block_rows == 128 && block_cols == 128;
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_fp8_type(typeQ) || !(row || col || tile))
    return SGEMM_ERR_INVALID_VALUE;
  if (!good_ld(ldx, cols) || !good_ld(ldq, cols) || !good_ld(lds, blocks_of(cols, block_cols)))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) {
    t_last_launches = 0;
    return SGEMM_SUCCESS;
  }
  if (!Q || !S) return SGEMM_ERR_INVALID_VALUE;
  QuantizeParams p = {};
  p.x = X;
  p.ldx = ldx;
  p.rows = rows;
  p.cols = cols;
  p.typeX = typeX;
  p.e5m2 = typeQ == SGEMM_TYPE_E5M2;
  p.tile = tile;
  (col ? p.qc : p.qr) = static_cast<unsigned char *>(Q);
  (col ? p.sc : p.sr) = S;
  (col ? p.ldqc : p.ldqr) = ldq;
  (col ? p.ldsc : p.ldsr) = lds;
  return quantize(p, block_rows, block_cols, false, reinterpret_cast<cudaStream_t>(stream));
}

sgemm_status_t sgemm_fp8_quantize_both(int64_t rows, int64_t cols, const void *X, sgemm_type_t typeX, int64_t ldx,
                                       sgemm_type_t typeQ, void *QR, int64_t ldqr, float *SR, int64_t ldsr, void *QC,
                                       int64_t ldqc, float *SC, int64_t ldsc, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_fp8_type(typeQ)) return SGEMM_ERR_INVALID_VALUE;
  if (!good_ld(ldx, cols) || !good_ld(ldqr, cols) || !good_ld(ldsr, blocks_of(cols, 128)) || !good_ld(ldqc, cols) ||
      !good_ld(ldsc, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) {
    t_last_launches = 0;
    return SGEMM_SUCCESS;
  }
  QuantizeParams p = {};
  p.x = X;
  p.ldx = ldx;
  p.rows = rows;
  p.cols = cols;
  p.typeX = typeX;
  p.e5m2 = typeQ == SGEMM_TYPE_E5M2;
  p.qr = static_cast<unsigned char *>(QR);
  p.sr = SR;
  p.ldqr = ldqr;
  p.ldsr = ldsr;
  p.qc = static_cast<unsigned char *>(QC);
  p.sc = SC;
  p.ldqc = ldqc;
  p.ldsc = ldsc;
  return quantize(p, 1, 128, true, reinterpret_cast<cudaStream_t>(stream));
}

sgemm_status_t sgemm_rms_norm_fp8(int64_t rows, int64_t cols, float eps, const void *X, int64_t ldx, const void *R,
                                  int64_t ldr, sgemm_type_t typeX, const void *W, sgemm_type_t typeW, void *H,
                                  int64_t ldh, void *Y, int64_t ldy, void *Q, sgemm_type_t typeQ, int64_t ldq,
                                  float *S, int64_t lds, float *T, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_fp8_type(typeQ)) return SGEMM_ERR_INVALID_VALUE;
  if ((typeW != typeX && typeW != SGEMM_TYPE_F32) || !(eps >= 0.0f)) return SGEMM_ERR_INVALID_VALUE;
  const int64_t kb = blocks_of(cols, SGEMM_FP8_BLOCK);
  if (!good_ld(ldx, cols) || (R && !good_ld(ldr, cols)) || (H && !good_ld(ldh, cols)) || (Y && !good_ld(ldy, cols)) ||
      !good_ld(ldq, cols) || !good_ld(lds, kb))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) {
    t_last_launches = 0;
    return SGEMM_SUCCESS;
  }
  const int e = type_size(typeX);
  const Range r[8] = {{X, rows, cols, ldx, e, false},      {R, R ? rows : 0, cols, ldr, e, false},
                      {W, 1, cols, cols, type_size(typeW), false},
                      {H, H ? rows : 0, cols, ldh, e, true}, {Y, Y ? rows : 0, cols, ldy, e, true},
                      {Q, rows, cols, ldq, 1, true},       {S, rows, kb, lds, 4, true},
                      {T, T ? 1 : 0, rows, rows, 4, true}};
  const sgemm_status_t st = check_ranges(r, 8);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  DeviceState *d = device_state(&why);
  if (!d) return why;
  NormParams p = {};
  p.x = X;
  p.r = R;
  p.w = W;
  p.h = H;
  p.y = Y;
  p.q = static_cast<unsigned char *>(Q);
  p.s = S;
  p.t = T;
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldh = ldh;
  p.ldy = ldy;
  p.ldq = ldq;
  p.lds = lds;
  p.rows = rows;
  p.cols = cols;
  p.typeX = typeX;
  p.w_f32 = typeW == SGEMM_TYPE_F32;
  p.e5m2 = typeQ == SGEMM_TYPE_E5M2;
  p.eps = eps;
  return queued(launch_rms_norm(p, d->sm_count, reinterpret_cast<cudaStream_t>(stream)), 1);
}

size_t sgemm_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || !good_dim(rows) || !good_dim(cols)) return 0;
  return static_cast<size_t>(norm_partials(rows, cols)) * static_cast<size_t>((cols + 7) / 8 * 8) * sizeof(float);
}

sgemm_status_t sgemm_rms_norm_backward(int64_t rows, int64_t cols, const void *DY, int64_t lddy, const void *H,
                                       int64_t ldh, sgemm_type_t typeX, const void *W, sgemm_type_t typeW,
                                       const float *T, const void *DH, int64_t lddh, void *DX, int64_t lddx, void *DW,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX)) return SGEMM_ERR_INVALID_VALUE;
  if (typeW != typeX && typeW != SGEMM_TYPE_F32) return SGEMM_ERR_INVALID_VALUE;
  if (!good_ld(lddy, cols) || !good_ld(ldh, cols) || (DH && !good_ld(lddh, cols)) || !good_ld(lddx, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (cols == 0 || (rows == 0 && !DW)) {
    t_last_launches = 0;
    return SGEMM_SUCCESS;
  }
  const size_t need = DW ? sgemm_rms_norm_backward_workspace(rows, cols) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return SGEMM_ERR_INVALID_VALUE;
  const int e = type_size(typeX);
  const Range r[8] = {{DY, rows, cols, lddy, e, false},
                      {H, rows, cols, ldh, e, false},
                      {W, rows ? 1 : 0, cols, cols, type_size(typeW), false},
                      {T, rows ? 1 : 0, rows, rows, 4, false},
                      {DH, DH ? rows : 0, cols, lddh, e, false},
                      {DX, rows, cols, lddx, e, true},
                      {DW, DW ? 1 : 0, cols, cols, type_size(typeW), true},
                      {workspace, need ? 1 : 0, static_cast<int64_t>(need / 4), static_cast<int64_t>(need / 4), 4, true}};
  const sgemm_status_t st = check_ranges(r, 8);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  if (!device_state(&why)) return why;
  NormGradParams p = {};
  p.dy = DY;
  p.h = H;
  p.w = W;
  p.dh = DH;
  p.t = T;
  p.dx = DX;
  p.dw = DW;
  p.partial = DW ? static_cast<float *>(workspace) : nullptr;
  p.lddy = lddy;
  p.ldh = ldh;
  p.lddh = lddh;
  p.lddx = lddx;
  p.rows = rows;
  p.cols = cols;
  p.typeX = typeX;
  p.w_f32 = typeW == SGEMM_TYPE_F32;
  return queued(launch_rms_norm_backward(p, reinterpret_cast<cudaStream_t>(stream)),
                (rows > 0 ? 1 : 0) + (DW ? 1 : 0));
}

}  // extern "C"
