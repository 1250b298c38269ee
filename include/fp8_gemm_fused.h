/*
 * fp8_gemm_fused.h -- products with a fused epilogue and the gated
 * feed-forward product, FP8 and BF16, with the BF16 backward passes.
 *
 * The conventions of fp8_gemm.h hold (device pointers owned by the caller,
 * work enqueued on `stream` of the current device, arguments validated before
 * anything is enqueued, deterministic results, an fp8g_status returned), with
 * these differences:
 *   - Nothing is allocated and no memory is kept between calls: the forward
 *     calls use no workspace, the backward calls the caller's, which may be
 *     reused as soon as the stream's work has passed it.  Calls on different
 *     streams do not interact as long as their workspaces and outputs differ.
 *   - No FP32 value is rounded before the outputs are, once, to BF16, except
 *     the gradients of the pre-activations, which are rounded to BF16 as the
 *     operands of the backward products.
 *   - BF16: K % 8 == 0, strides in elements, lda and ldb (and those of every
 *     other K-contiguous BF16 operand) multiples of 8.  FP8: K % 16 == 0,
 *     strides in bytes, as in fp8_gemm.h.
 *   - Residuals, output gradients and pre-activations may have any row stride
 *     >= N and any alignment of their element type; rows that start 16-byte
 *     aligned are read and written in 16-byte accesses.
 *   - An output (and the workspace) must not share memory with another output
 *     or an operand: such calls are refused with FP8G_ERR_ARG.  Rows of one may
 *     lie between rows of the other (column ranges of one buffer), operands
 *     may overlap each other, and the residual may be the output itself.
 *   - K = 0 gives Z = bias; M = 0 gives zero weight and bias gradients.
 *
 * Activations: z; max(z, 0); z / (1 + exp(-z)); z (1 + erf(z / sqrt 2)) / 2;
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2.  The slope of
 * FP8G_ACT_RELU at 0 is 0.
 */
#ifndef FP8_GEMM_FUSED_H
#define FP8_GEMM_FUSED_H

#include <stdint.h>

#include "fp8_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8G_ACT_NONE = 0,
    FP8G_ACT_RELU = 1,
    FP8G_ACT_SILU = 2,
    FP8G_ACT_GELU = 3,
    FP8G_ACT_GELU_TANH = 4
} fp8g_activation;

/*
 * FP8 product with a fused epilogue:
 *   Z[i][j] = scale_a[i] * scale_b[j] * sum_k A[i][k] B[j][k] + bias[j]
 *   D[i][j] = bf16_rne( act(Z[i][j]) + R[i][j] )
 *   A [M x K], B [N x K] FP8 codes, D [M x N] BF16: as for fp8_gemm_nt.
 *   scale_a: scale_a_n floats, scale_a_n = M (one per row) or 1; scale_b:
 *     scale_b_n floats, scale_b_n = N (one per output channel) or 1; either
 *     pointer NULL = 1.
 *   bias: [N] floats or NULL = 0.  Scales and bias 4-byte aligned.
 *   R: [M][ldr] BF16 or NULL = 0.  R may be D itself, with ldr = ldd; a matrix
 *     that overlaps D in another way is refused.
 * The kernel is chosen by an estimate of its time (fp8_gemm_fused_plan): for
 * few tokens or few output columns the swapped decode kernel (4 waves
 * splitting K over 16, 32 or 64 weight rows, tokens in tiles of up to 64), else
 * the LDS-tiled one with 128 x 128, 128 x 256 or 256 x 256 tiles.  The choice
 * never changes which elements are written.
 */
int fp8_gemm_nt_fused(const void *A, int64_t lda, int a_dtype, const void *B, int64_t ldb, int b_dtype,
                      const float *scale_a, int scale_a_n, const float *scale_b, int scale_b_n,
                      const float *bias, int activation, const void *R, int64_t ldr,
                      void *D, int64_t ldd, int M, int N, int K, void *stream);

/*
 * The same with BF16 operands and no scales.
 *   preact: [M][ldp] floats or NULL: receives Z (for the backward pass).
 */
int bf16_gemm_nt_fused(const void *A, int64_t lda, const void *B, int64_t ldb, const float *bias, int activation,
                       const void *R, int64_t ldr, void *D, int64_t ldd, float *preact, int64_t ldp,
                       int M, int N, int K, void *stream);

/*
 * Backward pass of bf16_gemm_nt_fused:
 *   dZ = G act'(Z)  (G: the gradient of D, [M][ldg] BF16; also that of R)
 *   dA = bf16_rne( dZ . B )     [M][ldda]
 *   dB = bf16_rne( dZ^T . A )   [N][lddb]
 *   dbias[j] = sum_i dZ[i][j]   [N] floats, of the FP32 dZ
 *   Each of dA, dB and dbias may be NULL (not computed).  ldda and lddb are
 *   multiples of 8; dA and dB 16-byte aligned.
 *   preact: Z, as kept by the forward call; NULL with FP8G_ACT_NONE only.
 *   workspace: at least bf16_gemm_nt_fused_backward_workspace(M, N, K) bytes,
 *   256-byte aligned; it holds dZ in BF16, the bias gradient's partial sums and,
 *   for products with few output tiles and a long sum, the FP32 sums of their
 *   splits over K (added in split order).
 */
int bf16_gemm_nt_fused_backward(const void *G, int64_t ldg, const void *A, int64_t lda, const void *B, int64_t ldb,
                                const float *preact, int64_t ldp, int activation,
                                void *dA, int64_t ldda, void *dB, int64_t lddb, float *dbias,
                                void *workspace, int64_t workspace_bytes, int M, int N, int K, void *stream);

/* Bytes of workspace of the call above (a negative fp8g_status for bad sizes). */
int64_t bf16_gemm_nt_fused_backward_workspace(int M, int N, int K);

/*
 * Gated feed-forward product (both projections, activation and product in one
 * kernel), FP8:
 *   P[i][j] = scale_a[i] * scale_g[j] * sum_k A[i][k] Wg[j][k]
 *   U[i][j] = scale_a[i] * scale_u[j] * sum_k A[i][k] Wu[j][k]
 *   D[i][j] = bf16_rne( act(P[i][j]) * U[i][j] )
 *   A [M x K], Wg and Wu [N x K] FP8 codes of one dtype (their strides may
 *   differ), D [M x N] BF16.  scale_a: scale_a_n floats (M or 1); scale_g and
 *   scale_u: scale_w_n floats each (N or 1); NULL = 1.
 */
int fp8_gated_nt(const void *A, int64_t lda, int a_dtype, const void *Wg, int64_t ldg, const void *Wu, int64_t ldu,
                 int w_dtype, const float *scale_a, int scale_a_n, const float *scale_g, const float *scale_u,
                 int scale_w_n, int activation, void *D, int64_t ldd, int M, int N, int K, void *stream);

/*
 * The same with BF16 operands and no scales.
 *   pre_g, pre_u: [M][ldp] floats, or both NULL: receive P and U.
 */
int bf16_gated_nt(const void *A, int64_t lda, const void *Wg, int64_t ldg, const void *Wu, int64_t ldu,
                  int activation, void *D, int64_t ldd, float *pre_g, float *pre_u, int64_t ldp,
                  int M, int N, int K, void *stream);

/*
 * Backward pass of bf16_gated_nt (G: the gradient of D, [M][ldgrad] BF16):
 *   dP = G U act'(P),  dU = G act(P)
 *   dA = bf16_rne( dP . Wg + dU . Wu )                      [M][ldda]
 *   dWg = bf16_rne( dP^T . A ),  dWu = bf16_rne( dU^T . A )  [N][lddw] each
 *   dA may be NULL; so may dWg and dWu, together.
 *   workspace: at least bf16_gated_nt_backward_workspace(M, N, K) bytes,
 *   256-byte aligned; it holds dP and dU in BF16 and the split sums, as above.
 */
int bf16_gated_nt_backward(const void *G, int64_t ldgrad, const void *A, int64_t lda, const void *Wg, int64_t ldg,
                           const void *Wu, int64_t ldu, const float *pre_g, const float *pre_u, int64_t ldp,
                           int activation, void *dA, int64_t ldda, void *dWg, void *dWu, int64_t lddw,
                           void *workspace, int64_t workspace_bytes, int M, int N, int K, void *stream);

/* Bytes of workspace of the call above (a negative fp8g_status for bad sizes). */
int64_t bf16_gated_nt_backward_workspace(int M, int N, int K);

/*
 * Kernel choice for a problem, without launching anything (host only).
 *   op: 0 = fp8_gemm_nt_fused, 1 = fp8_gated_nt, 2 = bf16_gemm_nt_fused,
 *   3 = bf16_gated_nt, 4 = one BF16 backward product (m x n outputs, reduced
 *   over k), with k_splits splits of k; 4 + FP8G_PLAN_PAIR = two of them in
 *   one launch (the weight gradients of bf16_gated_nt_backward: m = N, n = K,
 *   k = M), with the workgroups of both.
 * Fills the plan of fp8_gemm.h: variant 1 = tiled 256 x 256, 2 = tiled 128 x
 * 256, 7 = tiled 128 x 128 (m x n of the products; the gated forms' tiles hold
 * half as many output columns), 4 = swapped decode, 0 = nothing to launch;
 * tile_m and tile_n in rows and columns of D.
 */
#define FP8G_PLAN_PAIR 16
int fp8_gemm_fused_plan(int op, int m, int n, int k, fp8g_plan *out);

#ifdef __cplusplus
}
#endif

#endif /* FP8_GEMM_FUSED_H */
