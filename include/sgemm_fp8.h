/*
 * sgemm_fp8.h -- the linear layer in 8-bit floating point: the product of
 * block-scaled operands, the quantiser that makes them, and the RMS norm
 * (with the residual's addition) that feeds the product, with its gradient.
 * Part of the library declared in sgemm.h; its streams, status codes, device
 * status word, wait limit and argument checks apply here too.
 *
 * An 8-bit operand is a row-major matrix of E4M3 (largest value F = 448) or
 * E5M2 (F = 57344) elements together with one FP32 scale per block; an
 * element stands for q * s.  A block spans 128 elements along the inner
 * dimension of the product that reads it and 1 or 128 along the outer one; the
 * last blocks are cut at the matrix' edge.  The scales of a rows x cols matrix
 * with blocks of br x bc are a row-major ceil(rows / br) x ceil(cols / bc)
 * matrix.
 *
 * All pointers are device pointers on the current device, owned by the caller.
 * None of these calls allocates device memory, so every one of them may be
 * captured into a CUDA graph.  Outputs must not overlap inputs or each other
 * (SGEMM_ERR_ALIASING).  Leading dimensions count elements.  Rows whose start
 * is a multiple of 16 bytes take the fast paths; other layouts give the same
 * results.
 *
 * Arithmetic is FP32 throughout: every sum, norm and scale is held in 32 bits,
 * and a result is rounded once, where it is stored.  Subnormals are kept (of the
 * product of two scales, as FP32 holds them: see sgemm_fp8()).
 */
#ifndef DENSE_FP32_MATRIX_10_GB300_SGEMM_FP8_H_
#define DENSE_FP32_MATRIX_10_GB300_SGEMM_FP8_H_

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sgemm_type {
  SGEMM_TYPE_F32 = 0,
  SGEMM_TYPE_BF16 = 1,
  SGEMM_TYPE_F16 = 2,
  SGEMM_TYPE_E4M3 = 8, /* 1-4-3 bits, no infinity */
  SGEMM_TYPE_E5M2 = 9  /* 1-5-2 bits */
} sgemm_type_t;

/* Elements of a block along a product's inner dimension. */
#define SGEMM_FP8_BLOCK 128

/*
 * C = alpha * op(A) * op(B) + beta * C with 8-bit operands:
 *
 *   C[m,n] = alpha * sum_b SA(m,b) * SB(n,b) * sum_{k in block b} A(m,k) * B(k,n)
 *            + beta * C[m,n]
 *
 * op, M, N, K and the leading dimensions as in sgemm(): A is stored M x K
 * (transA = N) or K x M (T), B is stored K x N (N) or N x K (T).  blockA is the
 * extent, 1 or 128, of A's blocks along M; SA is then ceil(M / blockA) x
 * ceil(K / 128) for transA = N and ceil(K / 128) x ceil(M / blockA) for T,
 * row stride ldsa.  blockB is the extent of B's blocks along N; SB is
 * ceil(K / 128) x ceil(N / blockB) for transB = N and ceil(N / blockB) x
 * ceil(K / 128) for T.  typeA and typeB are E4M3 or E5M2, each its own;
 * typeC is F32, BF16 or F16.  A layer's forward product is N,T with blocks 1
 * and 128, its input gradient N,N with blocks 1 and 128, its weight gradient
 * T,N with blocks 1 and 1.
 *
 * Each block's products are summed on the tensor cores, then scaled and added
 * to the output's sum in FP32 registers.  The two scales of a block are
 * multiplied first, in FP32: where SA * SB is a normal number (2^-126 to
 * 2^128) the block counts in full.  Below, its part of C is off by up to
 * 2^-150 times its unscaled sum of magnitudes (2^-125 in all for E4M3 by E4M3,
 * 2^-111 for E5M2 by E5M2; a block of zeros still counts nothing); from 2^128
 * on it is an infinity, or NaN where the block's sum is zero.  Degenerate cases as in sgemm():
 * K == 0 or alpha == 0 give C = beta * C without reading A, B or the scales,
 * and beta == 0 never reads C.  One launch; deterministic.
 */
SGEMM_API sgemm_status_t sgemm_fp8(int transA, int transB, int64_t M, int64_t N, int64_t K,
                                   float alpha, const void *A, sgemm_type_t typeA, int64_t lda,
                                   const float *SA, int64_t ldsa, int blockA, const void *B,
                                   sgemm_type_t typeB, int64_t ldb, const float *SB, int64_t ldsb,
                                   int blockB, float beta, void *C, sgemm_type_t typeC, int64_t ldc,
                                   void *stream);

/* The forms of sgemm_fp8()'s kernel. */
typedef enum sgemm_fp8_form {
  SGEMM_FP8_FORM_FEW_16 = 0, /* up to 16 rows of C: 128 of its columns x 16 rows, one CTA or a cluster */
  SGEMM_FP8_FORM_FEW_32 = 1, /* up to 32 */
  SGEMM_FP8_FORM_FEW_64 = 2, /* up to 64 */
  SGEMM_FP8_FORM_HALF = 3,   /* 128 x 64, one CTA or a cluster */
  SGEMM_FP8_FORM_TILE = 4,   /* 128 x 128, one CTA or a cluster */
  SGEMM_FP8_FORM_LOADED = 5, /* the same, of operands that TMA cannot read */
  SGEMM_FP8_FORM_PAIR = 6,   /* 256 x 256 on two SMs, C written by the threads */
  SGEMM_FP8_FORM_PAIR_STAGED = 7, /* the same for rows of C off 16 bytes, through shared memory */
  SGEMM_FP8_FORM_PAIR_BULK = 8    /* the same with TMA stores */
} sgemm_fp8_form_t;

/*
 * The form that sgemm_fp8() would run for these arguments, or -1 if they are
 * invalid or nothing is multiplied; *split (if not NULL) is the number of CTAs
 * of a cluster that share the inner dimension of one tile.  Host only, as
 * sgemm_select_algo(); without a usable device, for 152 SMs.
 */
SGEMM_API int sgemm_fp8_select_form(int transA, int transB, int64_t M, int64_t N, int64_t K,
                                    const void *A, int64_t lda, const void *B, int64_t ldb,
                                    int blockB, float beta, const void *C, sgemm_type_t typeC,
                                    int64_t ldc, int *split);

/*
 * Quantises X (rows x cols; F32, BF16 or F16) in blocks of block_rows x
 * block_cols, which are 1 x 128, 128 x 1 or 128 x 128: with a the largest |x|
 * of a block,
 *
 *   s = max(a / F, 2^-126),    q = x / s rounded to nearest even.
 *
 * A block of zeros has q = 0 and the least scale.  A block that holds a NaN or
 * an infinity has that as its scale, so that whatever the product makes of it
 * is NaN.  Q is rows x cols (E4M3 or E5M2), S as described above.
 */
SGEMM_API sgemm_status_t sgemm_fp8_quantize(int64_t rows, int64_t cols, const void *X,
                                            sgemm_type_t typeX, int64_t ldx, void *Q,
                                            sgemm_type_t typeQ, int64_t ldq, float *S, int64_t lds,
                                            int block_rows, int block_cols, void *stream);

/*
 * The 1 x 128 and the 128 x 1 quantisation of X in one pass over it: QR, SR
 * and QC, SC are what sgemm_fp8_quantize() gives for either (the operands of
 * a gradient's two products).
 */
SGEMM_API sgemm_status_t sgemm_fp8_quantize_both(int64_t rows, int64_t cols, const void *X,
                                                 sgemm_type_t typeX, int64_t ldx,
                                                 sgemm_type_t typeQ, void *QR, int64_t ldqr,
                                                 float *SR, int64_t ldsr, void *QC, int64_t ldqc,
                                                 float *SC, int64_t ldsc, void *stream);

/*
 * RMS norm of x + r with an 8-bit output, row by row:
 *
 *   h = x + r,   t = 1 / sqrt(mean(h^2) + eps),   y = h * t * w,
 *   (q, s) = y quantised in 1 x 128 blocks (as sgemm_fp8_quantize(), but q is
 *            y * (1 / s) rounded: beside a middle of two 8-bit values, within
 *            2^-22 of it, that may be the other neighbour than for y / s)
 *
 * X and R (NULL: h = x) are rows x cols of typeX (F32, BF16, F16), W has cols
 * elements of typeW (F32 or typeX).  Q and S are always written; H and Y (of
 * typeX) and T (rows floats) where not NULL.  Neither h nor y is rounded before
 * the later steps; H and Y hold them rounded to typeX.  rows == 0 or cols == 0
 * do nothing (T is not written then either).
 */
SGEMM_API sgemm_status_t sgemm_rms_norm_fp8(int64_t rows, int64_t cols, float eps, const void *X,
                                            int64_t ldx, const void *R, int64_t ldr,
                                            sgemm_type_t typeX, const void *W, sgemm_type_t typeW,
                                            void *H, int64_t ldh, void *Y, int64_t ldy, void *Q,
                                            sgemm_type_t typeQ, int64_t ldq, float *S, int64_t lds,
                                            float *T, void *stream);

/*
 * Gradient of y = h * t * w with t = 1 / sqrt(mean(h^2) + eps) as the forward
 * pass wrote it: with g = dy * w,
 *
 *   dx = t * (g - h * t^2 * mean(g * h)) + dh,     dw = sum over rows of dy * h * t
 *
 * DY, H, DH and DX are rows x cols of typeX; DH (NULL: none) is the gradient
 * that reaches h along the residual path, and dx is the gradient of x and of
 * r alike.  DW (NULL: not computed) has cols elements of typeW.  The
 * quantisation of y is passed over (its gradient is taken as the identity).
 * workspace: sgemm_rms_norm_backward_workspace(rows, cols) bytes, 16-byte
 * aligned; it may be NULL when DW is NULL.  The rows' sums are added in a fixed
 * order, so results repeat bit for bit on one device.
 */
SGEMM_API sgemm_status_t sgemm_rms_norm_backward(int64_t rows, int64_t cols, const void *DY,
                                                 int64_t lddy, const void *H, int64_t ldh,
                                                 sgemm_type_t typeX, const void *W,
                                                 sgemm_type_t typeW, const float *T, const void *DH,
                                                 int64_t lddh, void *DX, int64_t lddx, void *DW,
                                                 void *workspace, size_t workspace_bytes,
                                                 void *stream);

/* Bytes of workspace that sgemm_rms_norm_backward() needs (0 for empty or
 * negative sizes).  Host only. */
SGEMM_API size_t sgemm_rms_norm_backward_workspace(int64_t rows, int64_t cols);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* DENSE_FP32_MATRIX_10_GB300_SGEMM_FP8_H_ */
