/*
 * fp8_gemm_experts.h -- experts' products over ragged groups of rows (BF16
 * with the backward pass, 8-bit integers), the dense product in 8-bit integers
 * with a fused epilogue, and the quantisation of token rows.
 *
 * The conventions of fp8_gemm.h hold (device pointers owned by the caller,
 * work enqueued on `stream` of the current device, arguments validated before
 * anything is enqueued, deterministic results, an fp8g_status returned), with
 * these differences:
 *   - Nothing is allocated, no workspace is used and no memory is kept between
 *     calls, so calls on different streams do not interact as long as their
 *     outputs differ, and any call may be captured into a graph.
 *   - Sums are held in 32 bits (FP32, or exact integers) and rounded to the
 *     output's type once.
 *   - BF16: strides in elements, multiples of 8; K % 8 == 0.  8-bit integers:
 *     strides in bytes, multiples of 16; K % 16 == 0 and K <= 131056, below
 *     which no sum of products of codes -128 .. 127 leaves 32 bits.
 *   - An output must not share memory with another output or an operand
 *     (FP8G_ERR_ARG), except the residual with the output itself.
 *
 * Ragged groups: G experts share M rows.  Expert g owns the rows offsets[g] ..
 * offsets[g + 1] - 1, any number of them (also none), starting anywhere;
 * offsets holds G + 1 int32 on the device, from 0 to M, and does not decrease.
 * Rows before offsets[0] and from offsets[G] on belong to no expert.  Values
 * outside 0 .. M count as the nearer end; where the offsets decrease, which of
 * the rows concerned are computed, and with which expert's weights, is not
 * defined, but nothing outside the matrices is read or written.  The host
 * never reads the offsets: the kernel is chosen from M and G.
 *   B: expert g's [N x K] weights begin b_stride elements after those of
 *   expert g - 1 (b_stride >= (N - 1) ldb + K and aligned as ldb is).
 *   N % 8 == 0 and N < 2^22, G <= 65535.
 *   At most 2^30 tiles of the chosen kernel (FP8G_ERR_SHAPE), which outputs that
 *   fit the memory do not reach.
 */
#ifndef FP8_GEMM_EXPERTS_H
#define FP8_GEMM_EXPERTS_H

#include <stdint.h>

#include "fp8_gemm_fused.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Ragged grouped product, BF16:
 *   D[r][n] = bf16_rne( sum_k A[r][k] B[g][n][k] )   for the rows r of expert g
 *   A [M][lda], D [M][ldd] BF16, 16-byte aligned; ldd at most (2^23 - 16) / 2,
 *   as every output's stride here.  Rows of no expert are neither read from A
 *   nor written to D.  K = 0 writes zeros.
 * Few rows per expert take the few-token kernel (16, 32 or 64 weight rows per
 * workgroup, tiles of 16, 32 or 64 rows of one expert), more the LDS-tiled one
 * (128 x 128, 128 x 256 or 256 x 256); the choice goes by an estimate of the
 * time (fp8_gemm_experts_plan) and never changes which elements are written.
 */
int bf16_grouped_gemm_ragged(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride,
                             const int32_t *offsets, void *D, int64_t ldd, int M, int G, int N, int K, void *stream);

/*
 * Its backward pass (dD: the gradient of D, [M][ldg] BF16, 16-byte aligned,
 * ldg a multiple of 8):
 *   dA[r] = bf16_rne( sum_n dD[r][n] B[g][n] )            [M][ldda], zeros for the rows of no expert
 *   dB[g] = bf16_rne( sum_{r of g} dD[r]^T A[r] )         [G][N][lddb], zeros for an expert without rows;
 *           expert g's begins db_stride elements after expert g - 1's
 *   Either of dA and dB may be NULL (not computed).  Rows of dD of no expert
 *   are not read.  M at most 2^30.
 */
int bf16_grouped_gemm_ragged_backward(const void *dD, int64_t ldg, const void *A, int64_t lda, const void *B,
                                      int64_t ldb, int64_t b_stride, const int32_t *offsets, void *dA, int64_t ldda,
                                      void *dB, int64_t lddb, int64_t db_stride, int M, int G, int N, int K,
                                      void *stream);

/*
 * Ragged grouped product in 8-bit integers:
 *   D[r][n] = bf16_rne( scale_a[r] * scale_b[g][n] * sum_k A[r][k] B[g][n][k] )
 *   A [M][lda], B int8, 16-byte aligned.  scale_a: [M] floats, one per row;
 *   scale_b: [G][N] floats, one per expert and channel; either NULL = 1.
 */
int int8_grouped_gemm_ragged(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride,
                             const float *scale_a, const float *scale_b, const int32_t *offsets, void *D, int64_t ldd,
                             int M, int G, int N, int K, void *stream);

/*
 * Product in 8-bit integers with a fused epilogue:
 *   Z[i][j] = scale_a[i] * scale_b[j] * sum_k A[i][k] B[j][k] + bias[j]
 *   D[i][j] = bf16_rne( act(Z[i][j]) + R[i][j] )
 *   A [M][lda], B [N][ldb] int8; everything else as for fp8_gemm_nt_fused.
 */
int int8_gemm_nt_fused(const void *A, int64_t lda, const void *B, int64_t ldb, const float *scale_a, int scale_a_n,
                       const float *scale_b, int scale_b_n, const float *bias, int activation, const void *R,
                       int64_t ldr, void *D, int64_t ldd, int M, int N, int K, void *stream);

/*
 * Quantisation of rows to 8-bit integers with a scale each:
 *   scale[m] = max_k |X[m][k]| / 127
 *   Q[m][k]  = 127 X[m][k] / max_k |X[m][k]|, rounded to the nearest whole
 *              number, halves to even (exactly: not by a rounded reciprocal)
 *   X [M][ldx] BF16 (16-byte aligned, ldx a multiple of 8), Q [M][ldq] int8
 *   (16-byte aligned, ldq a multiple of 16), K % 16 == 0.  A row of zeros, and
 *   every row of K = 0, has the scale 0; a row that holds an infinity or a NaN
 *   the scale NaN and codes 0.
 */
int int8_quantize_rows(const void *X, int64_t ldx, void *Q, int64_t ldq, float *scale, int M, int K, void *stream);

/*
 * Kernel choice for a problem, without launching anything (host only).
 *   op: 0 = bf16_grouped_gemm_ragged, 1 = int8_grouped_gemm_ragged, 2 = its
 *   BF16 token gradient (m x k, reduced over n), 3 = the weight gradients (n x
 *   k each, reduced over the expert's rows), 4 = int8_gemm_nt_fused without
 *   activation and residual (groups is not used).
 * Fills the plan of fp8_gemm.h as fp8_gemm_fused_plan does; workgroups counts
 * as many tiles as any offsets can need (the tiled kernels run them on at most
 * 256 persistent workgroups).  Variant 0: nothing is launched, as there is
 * nothing to compute or the call refuses the size (integers with K > 131056,
 * gradients of more than 2^30 rows, more tiles than a launch holds).
 */
int fp8_gemm_experts_plan(int op, int m, int n, int k, int groups, fp8g_plan *out);

#ifdef __cplusplus
}
#endif

#endif /* FP8_GEMM_EXPERTS_H */
