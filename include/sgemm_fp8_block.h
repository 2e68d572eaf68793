/*
 * sgemm_fp8_block.h -- what stands around the products of a gated block in
 * 8-bit floating point: the norms behind and in front of a block with its gate
 * and the scaled residual, the block's gated unit, the gradients of both, and
 * the change of kept rows into a weight gradient's operand.  Part of the
 * library declared in sgemm.h; types, blocks, quantisation, streams, aliasing
 * and alignment are as in sgemm_fp8.h.
 *
 * A checkpoint is what the forward pass keeps of a matrix for the backward
 * pass in 8 bits: its 1 x 128 quantisation as sgemm_fp8_quantize() defines it.
 * The gradients here take the matrix itself or its checkpoint (q, s), which
 * stands for q * s; the formulas are then of that value.  The quantisations'
 * own gradients are taken as the identity.  The outputs y, dg and du, which are
 * quantised as they are computed, are multiplied by 1 / s rounded: their x / s
 * has two FP32 roundings instead of one, so that one next to the middle of two
 * 8-bit values may become the other of them.
 *
 * None of these calls allocates device memory, all of them may be captured
 * into a CUDA graph, sums are held in FP32 and added in a fixed order, and
 * nothing is rounded before it is stored.
 */
#ifndef DENSE_FP32_MATRIX_10_GB300_SGEMM_FP8_BLOCK_H_
#define DENSE_FP32_MATRIX_10_GB300_SGEMM_FP8_BLOCK_H_

#include "sgemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The norm behind a block, its gate, the residual, and the norm in front of
 * the next block, row by row:
 *
 *   tp = 1 / sqrt(mean(a^2) + eps),     h = residual_scale * x + gate * (a * tp * wp)
 *   t  = 1 / sqrt(mean(h^2) + eps),     y = h * t * w,     (q, s) = y in 1 x 128 blocks
 *
 * A (the block's output) and X (the residual stream) are rows x cols of typeX
 * (F32, BF16, F16); WP and W have cols elements of typeW (F32 or typeX).  GATE
 * (NULL: 1) is ceil(rows / group_rows) x cols of typeGate (F32 or typeX): its
 * row r / group_rows goes with row r, so group_rows >= rows is one row for all,
 * and group_rows == 1 one for each.  Without a GATE, group_rows and typeGate
 * are not read.
 *
 * H (of typeX), Q and S are always written.  TP, T (rows floats each), QA with
 * SA (a's checkpoint) and QH with SH (h's) where not NULL, the checkpoints in
 * typeKeep (E4M3 or E5M2; not read without one).  h is rounded for H only.
 * rows == 0 or cols == 0 do nothing.
 */
SGEMM_API sgemm_status_t sgemm_sandwich_norm_fp8(
    int64_t rows, int64_t cols, float eps, float residual_scale, const void *A, int64_t lda, const void *X, int64_t ldx,
    sgemm_type_t typeX, const void *WP, const void *W, sgemm_type_t typeW, const void *GATE, int64_t ldgate,
    sgemm_type_t typeGate, int64_t group_rows, void *H, int64_t ldh, void *Q, sgemm_type_t typeQ, int64_t ldq, float *S,
    int64_t lds, float *TP, float *T, void *QA, int64_t ldqa, float *SA, int64_t ldsa, void *QH, int64_t ldqh, float *SH,
    int64_t ldsh, sgemm_type_t typeKeep, void *stream);

/*
 * Its gradient.  With DY the gradient of y, DH (NULL: none) the one that
 * reaches h along the residual path, and a, h, tp, t as the forward pass left
 * them:
 *
 *   g = dy * w,    H' = t * (g - h * t^2 * mean(g * h)) + dh,    dx = residual_scale * H'
 *   v = H' * gate * wp,    da = tp * (v - a * tp^2 * mean(v * a))
 *   dw = sum over rows of dy * h * t,       dwp = sum over rows of H' * gate * a * tp
 *   dgate = wp * (sum over the gate's rows of H' * a * tp)
 *
 * DY, DH, DA and DX are of typeX.  A and H are of typeX, or checkpoints of
 * typeA and typeH (E4M3 or E5M2) with their scales SA and SH, which are NULL
 * otherwise; the two are independent.  DWP, DW (cols elements of typeW) and
 * DGATE (as GATE) are computed where not NULL.  workspace:
 * sgemm_sandwich_norm_backward_workspace(rows, cols) bytes, 16-byte aligned; it
 * may be NULL when DWP, DW and DGATE are.  Sums over rows are added in a fixed
 * order: results repeat bit for bit.
 * With rows == 0 DWP and DW are zeros.
 */
SGEMM_API sgemm_status_t sgemm_sandwich_norm_backward(
    int64_t rows, int64_t cols, float residual_scale, const void *DY, int64_t lddy, const void *DH, int64_t lddh,
    sgemm_type_t typeX, const void *A, sgemm_type_t typeA, int64_t lda, const float *SA, int64_t ldsa, const void *H,
    sgemm_type_t typeH, int64_t ldh, const float *SH, int64_t ldsh, const void *WP, const void *W, sgemm_type_t typeW,
    const void *GATE, int64_t ldgate, sgemm_type_t typeGate, int64_t group_rows, const float *TP, const float *T,
    void *DA, int64_t ldda, void *DX, int64_t lddx, void *DWP, void *DW, void *DGATE, int64_t lddgate, void *workspace,
    size_t workspace_bytes, void *stream);

/* Bytes of workspace that sgemm_sandwich_norm_backward() needs (0 for empty or
 * negative sizes).  Host only. */
SGEMM_API size_t sgemm_sandwich_norm_backward_workspace(int64_t rows, int64_t cols);

/*
 * The gated unit y = g * p * u with p = 1 / (1 + exp(-g)), quantised in 1 x 128
 * blocks (the operand of the projection that follows).
 *
 * G and U are rows x cols of typeX (two halves of one product's output, say).
 * Q and S are always written, and where not NULL the checkpoints of g (QG, SG)
 * and u (QU, SU) in typeKeep.  y is not rounded before it is quantised.  Where
 * exp(-g) leaves FP32 (g < -87) p is 0.
 */
SGEMM_API sgemm_status_t sgemm_swiglu_fp8(int64_t rows, int64_t cols, const void *G, int64_t ldg, const void *U,
                                          int64_t ldu, sgemm_type_t typeX, void *Q, sgemm_type_t typeQ, int64_t ldq,
                                          float *S, int64_t lds, void *QG, int64_t ldqg, float *SG, int64_t ldsg,
                                          void *QU, int64_t ldqu, float *SU, int64_t ldsu, sgemm_type_t typeKeep,
                                          void *stream);

/*
 * Its gradient as the operands of the products that follow.  With DY (of typeX)
 * the gradient of y:
 *
 *   du = dy * g * p,     dg = dy * u * p * (1 + g * (1 - p)),     y = g * p * u
 *
 * G and U are of typeX, or checkpoints with their scales SG and SU (NULL
 * otherwise); typeG and typeU are the same.  With wide = cols rounded up to a
 * multiple of 128, [dg | du] is a rows x 2 wide matrix: dg in the columns
 * 0 .. cols - 1, du in wide .. wide + cols - 1, zeros behind each (zeros in QR
 * and QC, too, whatever the inputs hold).  It is quantised to typeZ in 1 x 128
 * blocks (QR; SR is rows x 2 wide / 128) and in 128 x 1 blocks (QC; SC is
 * ceil(rows / 128) x 2 wide); y, for the weight gradient of the projection
 * that read it, to typeY in 128 x 1 blocks (QY; SY is ceil(rows / 128) x cols).
 * All of them are written.
 */
SGEMM_API sgemm_status_t sgemm_swiglu_backward_fp8(
    int64_t rows, int64_t cols, const void *DY, int64_t lddy, sgemm_type_t typeX, const void *G, sgemm_type_t typeG,
    int64_t ldg, const float *SG, int64_t ldsg, const void *U, sgemm_type_t typeU, int64_t ldu, const float *SU,
    int64_t ldsu, sgemm_type_t typeZ, void *QR, int64_t ldqr, float *SR, int64_t ldsr, void *QC, int64_t ldqc, float *SC,
    int64_t ldsc, sgemm_type_t typeY, void *QY, int64_t ldqy, float *SY, int64_t ldsy, void *stream);

/*
 * The 128 x 1 quantisation of what a 1 x 128 quantisation (QX, SX) stands for
 * (q * s rounded to FP32): the operand of a weight gradient from the rows that
 * the forward pass multiplied with.
 */
SGEMM_API sgemm_status_t sgemm_fp8_requantize(int64_t rows, int64_t cols, const void *QX, sgemm_type_t typeX,
                                              int64_t ldqx, const float *SX, int64_t ldsx, void *Q, sgemm_type_t typeQ,
                                              int64_t ldq, float *S, int64_t lds, void *stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* DENSE_FP32_MATRIX_10_GB300_SGEMM_FP8_BLOCK_H_ */
