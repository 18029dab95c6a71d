/*
 * gemm_mxfp4.h -- products of libgemm_f32.so whose operands are held in
 * microscaled 4-bit floating point (MXFP4), and the conversions from and to
 * FP32.  Return codes, operand forms and error texts are those of
 * gemm_f32.h (gemm_f32_strerror, gemm_f32_last_error).
 *
 * Format.  A matrix of `rows` x `cols` values holds for every row r and
 * every block j of 32 columns, 32 j <= c < 32 (j + 1), one scale byte e and
 * 32 four-bit codes; the value at (r, c) is
 *
 *   2^(e - 127) * element(code),    e = 255: NaN, whatever the code,
 *
 * where bit 3 of a code is the sign and bits 2..0 select 0, 0.5, 1, 1.5, 2,
 * 3, 4 or 6.  This is the MXFP4 format (E2M1 elements, E8M0 scales) of the
 * Open Compute Project's microscaling formats specification 1.0.  Two codes
 * share a byte, the even column in the low half.
 *
 *   - A row of codes is ceil(cols / 32) whole blocks of 16 bytes.  Codes past
 *     `cols` in the last block must be zero (the conversions write zeros).
 *   - A row of scales is ceil(cols / 32) bytes, in storage of whole 4-byte
 *     words; the bytes past the last block are ignored (the conversions write
 *     zeros).
 *   - codes is 16-byte aligned with ld_codes and stride_codes multiples of
 *     16; scales is 4-byte aligned with ld_scales and stride_scales multiples
 *     of 4.  Other layouts are refused.
 *
 * Sizes (batch, rows, cols, M, N, K) are at most 2^31 - 1024.
 *
 * Scale bytes 253 and 254 can stand for values beyond FP32's range.  Read back,
 * such a value is infinite, and multiplied with FP32 infinite or NaN; a product
 * of two values in the format is exact, whatever their scales (255 aside), and
 * infinite only beyond FP32's range.
 *
 * Memory, streams, threads and errors are as in gemm_f32.h: device pointers
 * owned by the caller, nothing allocated, every argument checked before
 * anything is enqueued, results written only inside their rows and columns.
 * What overlaps is judged by address ranges, from an operand's first byte to the
 * last of its last row (of the last matrix of a batch).
 * The calls run on the device of `stream` (the current device for NULL).
 */
#ifndef GEMM_MXFP4_H
#define GEMM_MXFP4_H

#include <stdint.h>

#include "gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One matrix, or `batch` matrices a stride apart, in the format above. */
typedef struct gemm_mxfp4_matrix {
    void *codes;           /* row r at codes + r * ld_codes */
    int64_t ld_codes;      /* bytes; a multiple of 16, >= 16 ceil(cols / 32) */
    int64_t stride_codes;  /* bytes between matrices of a batch */
    void *scales;          /* row r at scales + r * ld_scales */
    int64_t ld_scales;     /* bytes; a multiple of 4, >= ceil(cols / 32) */
    int64_t stride_scales; /* bytes between matrices of a batch */
} gemm_mxfp4_matrix;

/*
 * gemm_mxfp4_quantize -- rounds FP32 matrices to the format, with blocks
 * along the rows (Q), along the columns (QT), or both in one read of X.
 *
 *   Q    rows x cols: the value of X[r][c], or NULL
 *   QT   cols x rows: the value of X[r][c] at row c, column r, or NULL
 *        (what a product needs that sums over X's rows); Q and QT not both
 *        NULL, not overlapping each other or X
 *   X    rows x cols, row-major FP32, ldx >= max(1, cols)
 *
 * For every block, with amax the largest magnitude in it:
 *
 *   e = clamp(floor(log2(amax)) - 2, -127, 127) + 127   (amax = 0: e = 0)
 *
 * and every code is the element nearest to x / 2^(e - 127), ties to the even
 * code, magnitudes above 6 to 6, the sign kept (of zeros and of values that
 * round to zero too).  A block that holds an infinity or a NaN has e = 255.
 *
 *   batch, strideX   `batch` matrices, X_b = X + b * strideX (floats);
 *                    strides of Q and QT must keep its matrices apart when
 *                    batch > 1
 *
 * rows == 0, cols == 0 or batch == 0 enqueues nothing.
 */
int gemm_mxfp4_quantize(int64_t batch, int64_t rows, int64_t cols,
                        const float *X, int64_t ldx, int64_t strideX,
                        const gemm_mxfp4_matrix *Q, const gemm_mxfp4_matrix *QT,
                        void *stream);

/*
 * gemm_mxfp4_dequantize -- writes the FP32 values of Q (rows x cols) to Y
 * (row-major, ldy >= max(1, cols)); exact, values beyond FP32 as infinities.
 * Batch as in gemm_mxfp4_quantize; matrices of Q may repeat (strides >= 0),
 * those of Y must not overlap.
 */
int gemm_mxfp4_dequantize(int64_t batch, int64_t rows, int64_t cols,
                          const gemm_mxfp4_matrix *Q,
                          float *Y, int64_t ldy, int64_t strideY,
                          void *stream);

/*
 * gemm_mxfp4 -- C_b = A_b x B_b^T with both operands in the format:
 *
 *   C[i][j] = sum over k < K of A[i][k] * B[j][k],   0 <= i < M, 0 <= j < N
 *
 *   A   M x K, B   N x K (blocks along k, the summed index, in both)
 *   C   M x N, row-major FP32, ldc >= max(1, N), not overlapping A or B
 *
 * Products are exact; they are summed in FP32 on the matrix cores, in an
 * order that depends only on the sizes, the row strides and on whether there
 * is a workspace.
 *
 *   batch        as in gemm_f32_strided_batched (strides of A and B >= 0, 0
 *                reuses one matrix; C's products must not overlap)
 *   workspace    NULL, or device memory of at least
 *                gemm_mxfp4_workspace_size(batch, M, N, K) bytes, 4-byte
 *                aligned, overlapping no operand, overwritten: a product with
 *                few output tiles and a long K is then computed as partial
 *                sums over slices of K that are added in a fixed order.  With
 *                NULL, K is never sliced.  Calls that overlap in time need
 *                workspaces of their own.
 *
 * M, N or batch == 0 enqueues nothing; K == 0 sets C to zero.
 */
int gemm_mxfp4(int64_t batch, int64_t M, int64_t N, int64_t K,
               const gemm_mxfp4_matrix *A, const gemm_mxfp4_matrix *B,
               float *C, int64_t ldc, int64_t strideC,
               void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace gemm_mxfp4 makes use of for these sizes (0: none, or
   invalid sizes). */
int64_t gemm_mxfp4_workspace_size(int64_t batch, int64_t M, int64_t N, int64_t K);

/*
 * gemm_mxfp4_weight -- C_b = A_b x op(W_b) with A in FP32 and W in the format:
 *
 *   opW = GEMM_F32_OP_T   W is N x K:  C[i][j] = sum over k of A[i][k] W[j][k]
 *                         (a stored layer applied to FP32 activations)
 *   opW = GEMM_F32_OP_N   W is K x N:  C[i][j] = sum over k of A[i][k] W[k][j]
 *                         (the gradient of the former with respect to its
 *                         activations: A the gradient of its output)
 *
 *   A   M x K, row-major FP32, lda >= max(1, K)
 *   C   M x N, row-major FP32, ldc >= max(1, N), not overlapping A or W
 *
 * A is not rounded: each of its values enters the product with its whole
 * significand (parts below 2^-133 in magnitude excepted), and the sums are
 * held in FP32.  Infinities and NaN in A propagate as in FP32.
 *
 * batch, workspace, and empty sizes as in gemm_mxfp4, with strideA >= 0 in
 * floats and gemm_mxfp4_weight_workspace_size.
 */
int gemm_mxfp4_weight(int opW, int64_t batch, int64_t M, int64_t N, int64_t K,
                      const float *A, int64_t lda, int64_t strideA,
                      const gemm_mxfp4_matrix *W,
                      float *C, int64_t ldc, int64_t strideC,
                      void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace gemm_mxfp4_weight makes use of for these arguments (0:
   none, or invalid ones). */
int64_t gemm_mxfp4_weight_workspace_size(int opW, int64_t batch, int64_t M, int64_t N, int64_t K);

/* Version of this header: 1. */
int gemm_mxfp4_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_MXFP4_H */
