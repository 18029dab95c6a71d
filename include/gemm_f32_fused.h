/*
 * gemm_f32_fused.h -- C ABI of the operators of libgemm_f32.so that do
 * something to a product of FP32 matrices while its sums are in registers: a
 * linear layer with bias, activation and residual, the softmax cross entropy
 * of tokens over a vocabulary, and the gradients of both.  MI355X (gfx950).
 *
 * Arithmetic: FP32 in, FP32 out, sums in FP32.  The products run on the 16-bit
 * matrix units, a value as the sum of parts that these take:
 *   - three bf16 parts, 24 bits, exactly (values below 2^-110 in magnitude are
 *     held to 2^-134), of whose nine products the six largest are summed: what is left
 *     out is at most 2^-23 of each |a b|, 2^-26 as a rule;
 *   - in large products with a workspace, where a look at every row of op(A)
 *     and column of op(B) finds the range for it, two fp16 parts of the value times a power of
 *     two for its row, of whose four products three are summed.  What that
 *     leaves out is at most 2^-21 of each |a b| (2^-24 as a rule), plus 2^-22
 *     of the sum of |a b|.  Whole numbers up to 2^11 are held exactly.  (Not in the
 *     products of the cross entropy's gradient: its probabilities have any range, and small
 *     ones beside a large one may be all that meets a value that isn't zero.)
 * A product that comes out infinite or NaN is computed again, with its tile, by
 * FP32 multiplies, so infinities, NaN and values next to the largest give what
 * gemm_f32 gives.  Few rows and small products may run on FP32 multiplies
 * throughout.  Activations and exponentials are evaluated in FP32.  Every call is
 * deterministic; how a sum is formed depends on the sizes, and in large products on
 * the ranges of the rows and columns that share a tile.
 *
 * Everything else is as in gemm_f32.h: row-major operands with leading
 * dimensions, device pointers aligned to 4 bytes, streams, ownership, errors
 * (GEMM_F32_OK, GEMM_F32_EINVAL, GEMM_F32_EHIP; gemm_f32_last_error has the
 * text).  Sizes are at most 2^31 - 1024, an operand spans at most 2^60 bytes.
 * Nothing is allocated: workspaces are the caller's (4-byte aligned, contents
 * don't matter, owned until the work has run; calls that may overlap need one
 * each).  An output must not overlap an input, another output or the workspace, except
 * where it is said (judged by address ranges, from an operand's first byte to its last); the
 * work runs on the stream's device.  Calls may be captured into a graph.
 */
#ifndef GEMM_F32_FUSED_H
#define GEMM_F32_FUSED_H

#include <stdint.h>

#include "gemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations. */
#define GEMM_F32_ACT_NONE 0
#define GEMM_F32_ACT_RELU 1      /* max(z, 0), slope 0 at 0; NaN stays NaN */
#define GEMM_F32_ACT_GELU 2      /* z (1 + erf(z / sqrt 2)) / 2 */
#define GEMM_F32_ACT_GELU_TANH 3 /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
#define GEMM_F32_ACT_SILU 4      /* z / (1 + exp(-z)) */

/*
 * What happens to a product's sums.
 *
 *   activation       GEMM_F32_ACT_*
 *   bias             N floats added to every row, or NULL; bias b of a batch
 *                    starts at bias + b * stride_bias (0: one for all)
 *   residual         M x N, added after the activation, or NULL; strides as
 *                    an operand's.  It may be C itself (same pointer, leading
 *                    dimension and stride): C = act(Z) + C.
 *   pre              M x N, receives Z = op(A) op(B) + bias for a backward
 *                    pass, or NULL
 */
typedef struct gemm_f32_epilogue {
    int activation;
    const float *bias;
    int64_t stride_bias;
    const float *residual;
    int64_t ld_residual, stride_residual;
    float *pre;
    int64_t ld_pre, stride_pre;
} gemm_f32_epilogue;

/*
 * gemm_f32_fused -- C_b = act(op(A_b) op(B_b) + bias_b) + R_b, 0 <= b < batch
 *
 * Operands, operand forms (GEMM_F32_OP_N, GEMM_F32_OP_T) and batches as in
 * gemm_f32_ex.  `epilogue` NULL: the bare product.
 *
 *   workspace    gemm_f32_fused_workspace_size bytes let a product with few
 *                tiles and a long K run in slices; NULL: it is not sliced.
 *
 * K == 0: Z is the bias, or zero.  M, N or batch 0: nothing is enqueued.
 */
int gemm_f32_fused(int opA, int opB, int64_t batch, int64_t M, int64_t N, int64_t K,
                   const float *A, int64_t lda, int64_t strideA,
                   const float *B, int64_t ldb, int64_t strideB,
                   const gemm_f32_epilogue *epilogue,
                   float *C, int64_t ldc, int64_t strideC,
                   void *workspace, int64_t workspace_bytes, void *stream);
/* 0 where no workspace helps, or where a size or form is invalid. */
int64_t gemm_f32_fused_workspace_size(int opA, int opB, int64_t batch, int64_t M, int64_t N,
                                      int64_t K);

/*
 * gemm_f32_fused_grad -- the gradients of gemm_f32_fused, from dC, the
 * gradient of its C:
 *
 *   dZ = dC act'(Z)
 *   dA = dZ op(B)^T, dB = op(A)^T dZ    each laid out as A and B are
 *   dbias = the sums of dZ's columns
 *
 * (the residual's gradient is dC).  dA, dB and dbias may each be NULL: not
 * computed; A is read for dB only and B for dA only.
 *
 *   pre              Z as gemm_f32_fused kept it; not read for ACT_NONE.
 *                    dC and pre have strides of their own.
 *   opA, opB         the forms the forward call had; dA is K x M for
 *                    GEMM_F32_OP_T, dB is N x K
 *   batch            gradients are per product: dA_b, dB_b and dbias_b.  A
 *                    gradient that is shared by a batch (an operand with
 *                    stride 0) is the caller's sum, or one product of
 *                    the stacked rows.  stride_dbias is at least N where
 *                    batch > 1.
 *   workspace        gemm_f32_fused_grad_workspace_size bytes (for the outputs
 *                    asked for); less is refused.
 *
 * M, N or K may be 0: dB and dbias are zero where M is 0, dA where N is.
 */
int gemm_f32_fused_grad(int opA, int opB, int64_t batch, int64_t M, int64_t N, int64_t K,
                        const float *dC, int64_t lddc, int64_t stride_dC,
                        int activation, const float *pre, int64_t ld_pre, int64_t stride_pre,
                        const float *A, int64_t lda, int64_t strideA,
                        const float *B, int64_t ldb, int64_t strideB,
                        float *dA, int64_t ldda, int64_t stride_dA,
                        float *dB, int64_t lddb, int64_t stride_dB,
                        float *dbias, int64_t stride_dbias,
                        void *workspace, int64_t workspace_bytes, void *stream);
/* want_*: whether that output will be asked for. */
int64_t gemm_f32_fused_grad_workspace_size(int opA, int opB, int64_t batch, int64_t M, int64_t N,
                                           int64_t K, int activation, int want_dA, int want_dB,
                                           int want_dbias);

/*
 * gemm_f32_cross_entropy -- softmax cross entropy of T tokens over a
 * vocabulary of V, from their hidden states and the output layer:
 *
 *   logit[t][v] = X[t] . W[v]
 *   lse[t]      = log sum over v of exp(logit[t][v])
 *   loss[t]     = lse[t] - logit[t][target[t]]
 *
 *   X, ldx       T x K
 *   W, ldw       V x K, V >= 1 (unless T is 0)
 *   target       T word numbers.  A token whose target is `ignore_index` (any
 *                value, usually negative) takes no part: its loss is 0, and its
 *                lse is only defined where its row of X and all its logits are finite
 *                and X and W stay below 3.38e38 (a tile is not computed again for
 *                it: padding of any values costs nothing).  Any other target
 *                outside [0, V) gives a loss of NaN.
 *   loss, lse    T floats each; either may be NULL.  A logit of +inf makes its
 *                token's lse +inf, and the loss too (NaN where it is the target's); one
 *                of -inf is no word; NaN makes both NaN.
 *   workspace    gemm_f32_cross_entropy_workspace_size bytes; less is refused
 *
 * The logits are not kept: each tile of them ends as a maximum and a sum of
 * exponentials a row.
 */
int gemm_f32_cross_entropy(int64_t T, int64_t V, int64_t K,
                           const float *X, int64_t ldx, const float *W, int64_t ldw,
                           const int64_t *target, int64_t ignore_index,
                           float *loss, float *lse,
                           void *workspace, int64_t workspace_bytes, void *stream);
int64_t gemm_f32_cross_entropy_workspace_size(int64_t T, int64_t V, int64_t K);

/*
 * gemm_f32_cross_entropy_grad -- the same, with the gradients of the sum over
 * t of grad_loss[t] loss[t]:
 *
 *   P[t][v] = grad_loss[t] (exp(logit[t][v] - lse[t]) - (v == target[t]))
 *   dX = P W (T x K), dW = P^T X (V x K)
 *
 *   grad_loss    T floats, or NULL for ones
 *   dX, dW       either may be NULL: not computed; dW is overwritten
 *   loss, lse    as above, either may be NULL
 *   workspace    holds the logits of as many tokens at a time as fit, so what
 *                it must hold does not grow with T x V:
 *                gemm_f32_cross_entropy_grad_workspace_size bytes are what is
 *                quickest (a few GiB at most, unless a single row's logits
 *                take more), gemm_f32_cross_entropy_grad_workspace_least the
 *                fewest that are accepted.  With anything less than the quickest no product
 *                runs in slices or fp16 parts.
 *
 * An ignored token's row of P, and so of dX, is zero, and its row of X takes
 * no part in dW even where it holds infinities or NaN.  A target that is
 * neither ignored nor in [0, V) makes its row of dX, and dW, NaN.
 */
int gemm_f32_cross_entropy_grad(int64_t T, int64_t V, int64_t K,
                                const float *X, int64_t ldx, const float *W, int64_t ldw,
                                const int64_t *target, int64_t ignore_index,
                                const float *grad_loss, float *loss, float *lse,
                                float *dX, int64_t lddx, float *dW, int64_t lddw,
                                void *workspace, int64_t workspace_bytes, void *stream);
int64_t gemm_f32_cross_entropy_grad_workspace_size(int64_t T, int64_t V, int64_t K);
int64_t gemm_f32_cross_entropy_grad_workspace_least(int64_t T, int64_t V, int64_t K);

/* 1 */
int gemm_f32_fused_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_FUSED_H */
