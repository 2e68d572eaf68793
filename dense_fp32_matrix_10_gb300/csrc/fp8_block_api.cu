// fp8_block_api.cu -- the C ABI of include/sgemm_fp8_block.h: argument checks
// (all on the host, before anything is queued), the degenerate cases and the
// dispatch.
#include "sgemm_fp8_block.h"

#include "dispatch.h"
#include "fp8_block.h"
#include "fp8_checks.h"

namespace sg {
namespace {

// Weights and gates: F32 or the call's type.
bool is_weight_type(int t, int typeX) { return t == typeX || t == SGEMM_TYPE_F32; }

// A matrix or its checkpoint: the type fits the scales (an empty one's may be null), and so do the strides.
bool good_kept(int type, int typeX, int64_t ld, const float *s, int64_t lds, int64_t rows, int64_t cols) {
  if (!good_ld(ld, cols)) return false;
  if (s) return is_fp8_type(type) && good_ld(lds, blocks_of(cols, SGEMM_FP8_BLOCK));
  return type == typeX || (is_fp8_type(type) && (rows == 0 || cols == 0));
}
Kept kept(const void *p, int type, int64_t ld, const float *s, int64_t lds) {
  return {p, s, ld, lds, type == SGEMM_TYPE_E5M2};
}

sgemm_status_t nothing() {
  t_last_launches = 0;
  return SGEMM_SUCCESS;
}

unsigned group_of(int64_t group_rows, int64_t rows) {
  return static_cast<unsigned>(group_rows < rows ? group_rows : rows);
}

// (The row stride of a single row says nothing about its alignment.)
Gate gate_of(const void *p, int64_t ld, unsigned group, int64_t rows, sgemm_type_t type) {
  return {p, group >= rows ? 0 : ld, group, p && type == SGEMM_TYPE_F32};
}

}  // namespace

}  // namespace sg

using namespace sg;

extern "C" {

sgemm_status_t sgemm_sandwich_norm_fp8(
    int64_t rows, int64_t cols, float eps, float residual_scale, const void *A, int64_t lda, const void *X, int64_t ldx,
    sgemm_type_t typeX, const void *WP, const void *W, sgemm_type_t typeW, const void *GATE, int64_t ldgate,
    sgemm_type_t typeGate, int64_t group_rows, void *H, int64_t ldh, void *Q, sgemm_type_t typeQ, int64_t ldq, float *S,
    int64_t lds, float *TP, float *T, void *QA, int64_t ldqa, float *SA, int64_t ldsa, void *QH, int64_t ldqh, float *SH,
    int64_t ldsh, sgemm_type_t typeKeep, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_fp8_type(typeQ) || !is_weight_type(typeW, typeX))
    return SGEMM_ERR_INVALID_VALUE;
  if (!(eps >= 0.0f) || (GATE && (!is_weight_type(typeGate, typeX) || group_rows < 1 || !good_ld(ldgate, cols))))
    return SGEMM_ERR_INVALID_VALUE;
  const int64_t kb = blocks_of(cols, SGEMM_FP8_BLOCK);
  if (!good_ld(lda, cols) || !good_ld(ldx, cols) || !good_ld(ldh, cols) || !good_ld(ldq, cols) || !good_ld(lds, kb))
    return SGEMM_ERR_INVALID_VALUE;
  if (!QA != !SA || !QH != !SH || ((QA || QH) && !is_fp8_type(typeKeep))) return SGEMM_ERR_INVALID_VALUE;
  if ((QA && (!good_ld(ldqa, cols) || !good_ld(ldsa, kb))) || (QH && (!good_ld(ldqh, cols) || !good_ld(ldsh, kb))))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return nothing();
  const int e = type_size(typeX);
  const unsigned group = GATE ? group_of(group_rows, rows) : 1;
  const Range r[] = {{A, rows, cols, lda, e, false},
                     {X, rows, cols, ldx, e, false},
                     {WP, 1, cols, cols, type_size(typeW), false},
                     {W, 1, cols, cols, type_size(typeW), false},
                     {GATE, GATE ? (rows + group - 1) / group : 0, cols, ldgate, GATE ? type_size(typeGate) : 1, false},
                     {H, rows, cols, ldh, e, true},
                     {Q, rows, cols, ldq, 1, true},
                     {S, rows, kb, lds, 4, true},
                     {TP, TP ? 1 : 0, rows, rows, 4, true},
                     {T, T ? 1 : 0, rows, rows, 4, true},
                     {QA, QA ? rows : 0, cols, ldqa, 1, true},
                     {SA, QA ? rows : 0, kb, ldsa, 4, true},
                     {QH, QH ? rows : 0, cols, ldqh, 1, true},
                     {SH, QH ? rows : 0, kb, ldsh, 4, true}};
  const sgemm_status_t st = check_ranges(r);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  DeviceState *d = device_state(&why);
  if (!d) return why;
  SandwichParams p = {};
  p.a = A;
  p.x = X;
  p.wp = WP;
  p.w = W;
  p.gate = gate_of(GATE, ldgate, group, rows, typeGate);
  p.h = H;
  p.q = static_cast<unsigned char *>(Q);
  p.qa = static_cast<unsigned char *>(QA);
  p.qh = static_cast<unsigned char *>(QH);
  p.s = S;
  p.sa = SA;
  p.sh = SH;
  p.tp = TP;
  p.t = T;
  p.lda = lda;
  p.ldx = ldx;
  p.ldh = ldh;
  p.ldq = ldq;
  p.lds = lds;
  p.ldqa = ldqa;
  p.ldsa = ldsa;
  p.ldqh = ldqh;
  p.ldsh = ldsh;
  p.rows = rows;
  p.cols = cols;
  p.w_f32 = typeW == SGEMM_TYPE_F32;
  p.e5m2 = typeQ == SGEMM_TYPE_E5M2;
  p.keep_e5m2 = typeKeep == SGEMM_TYPE_E5M2;
  p.eps = eps;
  p.residual_scale = residual_scale;
  const auto launch = typeX == SGEMM_TYPE_F32    ? launch_sandwich_norm_f32
                      : typeX == SGEMM_TYPE_BF16 ? launch_sandwich_norm_bf16
                                                 : launch_sandwich_norm_f16;
  return queued(launch(p, d->sm_count, reinterpret_cast<cudaStream_t>(stream)), 1);
}

size_t sgemm_sandwich_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || !good_dim(rows) || !good_dim(cols)) return 0;
  return static_cast<size_t>(sandwich_partials(rows, cols)) * sizeof(float);
}

sgemm_status_t sgemm_sandwich_norm_backward(
    int64_t rows, int64_t cols, float residual_scale, const void *DY, int64_t lddy, const void *DH, int64_t lddh,
    sgemm_type_t typeX, const void *A, sgemm_type_t typeA, int64_t lda, const float *SA, int64_t ldsa, const void *H,
    sgemm_type_t typeH, int64_t ldh, const float *SH, int64_t ldsh, const void *WP, const void *W, sgemm_type_t typeW,
    const void *GATE, int64_t ldgate, sgemm_type_t typeGate, int64_t group_rows, const float *TP, const float *T,
    void *DA, int64_t ldda, void *DX, int64_t lddx, void *DWP, void *DW, void *DGATE, int64_t lddgate, void *workspace,
    size_t workspace_bytes, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_weight_type(typeW, typeX))
    return SGEMM_ERR_INVALID_VALUE;
  if (!good_kept(typeA, typeX, lda, SA, ldsa, rows, cols) || !good_kept(typeH, typeX, ldh, SH, ldsh, rows, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (!good_ld(lddy, cols) || (DH && !good_ld(lddh, cols)) || !good_ld(ldda, cols) || !good_ld(lddx, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (GATE && (!is_weight_type(typeGate, typeX) || group_rows < 1 || !good_ld(ldgate, cols))) return SGEMM_ERR_INVALID_VALUE;
  if (DGATE && (!GATE || !good_ld(lddgate, cols))) return SGEMM_ERR_INVALID_VALUE;
  if (cols == 0 || (rows == 0 && !DWP && !DW)) return nothing();
  const bool sums = DWP || DW || DGATE;
  const size_t need = sums ? sgemm_sandwich_norm_backward_workspace(rows, cols) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
    return SGEMM_ERR_INVALID_VALUE;
  const int e = type_size(typeX), ew = type_size(typeW), eg = GATE ? type_size(typeGate) : 1;
  const unsigned group = GATE && rows ? group_of(group_rows, rows) : 1;
  const int64_t groups = GATE ? (rows + group - 1) / group : 0, kb = blocks_of(cols, SGEMM_FP8_BLOCK), one = rows ? 1 : 0;
  const int64_t floats = static_cast<int64_t>(need / 4);
  const Range r[] = {{DY, rows, cols, lddy, e, false},
                     {DH, DH ? rows : 0, cols, lddh, e, false},
                     {A, rows, cols, lda, type_size(typeA), false},
                     {SA, SA ? rows : 0, kb, ldsa, 4, false},
                     {H, rows, cols, ldh, type_size(typeH), false},
                     {SH, SH ? rows : 0, kb, ldsh, 4, false},
                     {WP, one, cols, cols, ew, false},
                     {W, one, cols, cols, ew, false},
                     {GATE, groups, cols, ldgate, eg, false},
                     {TP, one, rows, rows, 4, false},
                     {T, one, rows, rows, 4, false},
                     {DA, rows, cols, ldda, e, true},
                     {DX, rows, cols, lddx, e, true},
                     {DWP, DWP ? 1 : 0, cols, cols, ew, true},
                     {DW, DW ? 1 : 0, cols, cols, ew, true},
                     {DGATE, DGATE ? groups : 0, cols, lddgate, eg, true},
                     {workspace, need ? 1 : 0, floats, floats, 4, true}};
  const sgemm_status_t st = check_ranges(r);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  DeviceState *d = device_state(&why);
  if (!d) return why;
  SandwichGradParams p = {};
  p.dy = DY;
  p.dh = DH;
  p.wp = WP;
  p.w = W;
  p.a = kept(A, typeA, lda, SA, ldsa);
  p.h = kept(H, typeH, ldh, SH, ldsh);
  p.gate = gate_of(GATE, ldgate, group, rows, typeGate);
  p.tp = TP;
  p.t = T;
  p.da = DA;
  p.dx = DX;
  p.dwp = DWP;
  p.dw = DW;
  p.dgate = rows > 0 ? DGATE : nullptr;
  p.partial = sums ? static_cast<float *>(workspace) : nullptr;
  p.lddy = lddy;
  p.lddh = lddh;
  p.ldda = ldda;
  p.lddx = lddx;
  p.lddgate = group >= rows ? 0 : lddgate;
  p.rows = rows;
  p.cols = cols;
  p.typeX = typeX;
  p.w_f32 = typeW == SGEMM_TYPE_F32;
  p.residual_scale = residual_scale;
  p.wait_budget_ns = g_wait_budget_ns.load(std::memory_order_relaxed);
  p.status = d->status;
  int launches = 0;
  const cudaError_t err = launch_sandwich_norm_backward(p, reinterpret_cast<cudaStream_t>(stream), &launches);
  return queued(err, launches);
}

sgemm_status_t sgemm_swiglu_fp8(int64_t rows, int64_t cols, const void *G, int64_t ldg, const void *U, int64_t ldu,
                                sgemm_type_t typeX, void *Q, sgemm_type_t typeQ, int64_t ldq, float *S, int64_t lds,
                                void *QG, int64_t ldqg, float *SG, int64_t ldsg, void *QU, int64_t ldqu, float *SU,
                                int64_t ldsu, sgemm_type_t typeKeep, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_fp8_type(typeQ)) return SGEMM_ERR_INVALID_VALUE;
  const int64_t kb = blocks_of(cols, SGEMM_FP8_BLOCK);
  if (!good_ld(ldg, cols) || !good_ld(ldu, cols) || !good_ld(ldq, cols) || !good_ld(lds, kb)) return SGEMM_ERR_INVALID_VALUE;
  if (!QG != !SG || !QU != !SU || ((QG || QU) && !is_fp8_type(typeKeep))) return SGEMM_ERR_INVALID_VALUE;
  if ((QG && (!good_ld(ldqg, cols) || !good_ld(ldsg, kb))) || (QU && (!good_ld(ldqu, cols) || !good_ld(ldsu, kb))))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return nothing();
  const int e = type_size(typeX);
  const Range r[] = {{G, rows, cols, ldg, e, false},         {U, rows, cols, ldu, e, false},
                     {Q, rows, cols, ldq, 1, true},          {S, rows, kb, lds, 4, true},
                     {QG, QG ? rows : 0, cols, ldqg, 1, true}, {SG, QG ? rows : 0, kb, ldsg, 4, true},
                     {QU, QU ? rows : 0, cols, ldqu, 1, true}, {SU, QU ? rows : 0, kb, ldsu, 4, true}};
  const sgemm_status_t st = check_ranges(r);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  if (!device_state(&why)) return why;
  SwigluParams p = {};
  p.g = G;
  p.u = U;
  p.q = static_cast<unsigned char *>(Q);
  p.qg = static_cast<unsigned char *>(QG);
  p.qu = static_cast<unsigned char *>(QU);
  p.s = S;
  p.sg = SG;
  p.su = SU;
  p.ldg = ldg;
  p.ldu = ldu;
  p.ldq = ldq;
  p.lds = lds;
  p.ldqg = ldqg;
  p.ldsg = ldsg;
  p.ldqu = ldqu;
  p.ldsu = ldsu;
  p.rows = rows;
  p.cols = cols;
  p.typeX = typeX;
  p.e5m2 = typeQ == SGEMM_TYPE_E5M2;
  p.keep_e5m2 = typeKeep == SGEMM_TYPE_E5M2;
  return queued(launch_swiglu(p, reinterpret_cast<cudaStream_t>(stream)), 1);
}

sgemm_status_t sgemm_swiglu_backward_fp8(
    int64_t rows, int64_t cols, const void *DY, int64_t lddy, sgemm_type_t typeX, const void *G, sgemm_type_t typeG,
    int64_t ldg, const float *SG, int64_t ldsg, const void *U, sgemm_type_t typeU, int64_t ldu, const float *SU,
    int64_t ldsu, sgemm_type_t typeZ, void *QR, int64_t ldqr, float *SR, int64_t ldsr, void *QC, int64_t ldqc, float *SC,
    int64_t ldsc, sgemm_type_t typeY, void *QY, int64_t ldqy, float *SY, int64_t ldsy, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_float_type(typeX) || !is_fp8_type(typeZ) || !is_fp8_type(typeY))
    return SGEMM_ERR_INVALID_VALUE;
  const int64_t kb = blocks_of(cols, SGEMM_FP8_BLOCK), wide = 2 * kb * SGEMM_FP8_BLOCK, rb = blocks_of(rows, SGEMM_FP8_BLOCK);
  if (!good_dim(wide) || !SG != !SU || typeG != typeU || !good_kept(typeG, typeX, ldg, SG, ldsg, rows, cols) ||
      !good_kept(typeU, typeX, ldu, SU, ldsu, rows, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (!good_ld(lddy, cols) || !good_ld(ldqr, wide) || !good_ld(ldsr, 2 * kb) || !good_ld(ldqc, wide) ||
      !good_ld(ldsc, wide) || !good_ld(ldqy, cols) || !good_ld(ldsy, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return nothing();
  const Range r[] = {{DY, rows, cols, lddy, type_size(typeX), false},
                     {G, rows, cols, ldg, type_size(typeG), false},
                     {SG, SG ? rows : 0, kb, ldsg, 4, false},
                     {U, rows, cols, ldu, type_size(typeU), false},
                     {SU, SU ? rows : 0, kb, ldsu, 4, false},
                     {QR, rows, wide, ldqr, 1, true},
                     {SR, rows, 2 * kb, ldsr, 4, true},
                     {QC, rows, wide, ldqc, 1, true},
                     {SC, rb, wide, ldsc, 4, true},
                     {QY, rows, cols, ldqy, 1, true},
                     {SY, rb, cols, ldsy, 4, true}};
  const sgemm_status_t st = check_ranges(r);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  const DeviceState *d = device_state(&why);
  if (!d) return why;
  SwigluGradParams p = {};
  p.dy = DY;
  p.g = kept(G, typeG, ldg, SG, ldsg);
  p.u = kept(U, typeU, ldu, SU, ldsu);
  p.qr = static_cast<unsigned char *>(QR);
  p.qc = static_cast<unsigned char *>(QC);
  p.qy = static_cast<unsigned char *>(QY);
  p.sr = SR;
  p.sc = SC;
  p.sy = SY;
  p.lddy = lddy;
  p.ldqr = ldqr;
  p.ldsr = ldsr;
  p.ldqc = ldqc;
  p.ldsc = ldsc;
  p.ldqy = ldqy;
  p.ldsy = ldsy;
  p.rows = rows;
  p.cols = cols;
  p.z_e5m2 = typeZ == SGEMM_TYPE_E5M2;
  p.y_e5m2 = typeY == SGEMM_TYPE_E5M2;
  const auto launch = typeX == SGEMM_TYPE_F32    ? launch_swiglu_backward_f32
                      : typeX == SGEMM_TYPE_BF16 ? launch_swiglu_backward_bf16
                                                 : launch_swiglu_backward_f16;
  return queued(launch(p, d->sm_count, reinterpret_cast<cudaStream_t>(stream)), 1);
}

sgemm_status_t sgemm_fp8_requantize(int64_t rows, int64_t cols, const void *QX, sgemm_type_t typeX, int64_t ldqx,
                                    const float *SX, int64_t ldsx, void *Q, sgemm_type_t typeQ, int64_t ldq, float *S,
                                    int64_t lds, void *stream) {
  if (!good_dim(rows) || !good_dim(cols) || !is_fp8_type(typeX) || !is_fp8_type(typeQ)) return SGEMM_ERR_INVALID_VALUE;
  const int64_t kb = blocks_of(cols, SGEMM_FP8_BLOCK), rb = blocks_of(rows, SGEMM_FP8_BLOCK);
  if (!good_ld(ldqx, cols) || !good_ld(ldsx, kb) || !good_ld(ldq, cols) || !good_ld(lds, cols))
    return SGEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return nothing();
  const Range r[] = {{QX, rows, cols, ldqx, 1, false},
                     {SX, rows, kb, ldsx, 4, false},
                     {Q, rows, cols, ldq, 1, true},
                     {S, rb, cols, lds, 4, true}};
  const sgemm_status_t st = check_ranges(r);
  if (st != SGEMM_SUCCESS) return st;
  sgemm_status_t why = SGEMM_SUCCESS;
  if (!device_state(&why)) return why;
  RequantizeParams p = {};
  p.x = static_cast<const unsigned char *>(QX);
  p.sx = SX;
  p.q = static_cast<unsigned char *>(Q);
  p.s = S;
  p.ldx = ldqx;
  p.ldsx = ldsx;
  p.ldq = ldq;
  p.lds = lds;
  p.rows = rows;
  p.cols = cols;
  p.x_e5m2 = typeX == SGEMM_TYPE_E5M2;
  p.e5m2 = typeQ == SGEMM_TYPE_E5M2;
  return queued(launch_requantize(p, reinterpret_cast<cudaStream_t>(stream)), 1);
}

}  // extern "C"
