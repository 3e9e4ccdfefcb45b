/*
 * dq4_int8 — layers with 8-bit weights beside the 4-bit ones of dq4.h, for NVIDIA GB300
 * (compute capability 10.3): the row quantizer of LLM.int8 with its outlier columns, the
 * 8-bit matrix product, the gradient of its input, and a mixture-of-experts layer for few
 * tokens.
 *
 * Conventions are those of dq4.h: DEVICE pointers owned by the caller, no allocation and
 * no synchronization inside, work enqueued on `stream`, a status code returned (nothing is
 * enqueued on an error other than DQ4_ERR_LAUNCH), host threads may call concurrently, but
 * calls that share a workspace one at a time: most take several launches, which have to follow
 * each other in the stream.
 * Element types are DQ4_OUT_F16 / DQ4_OUT_BF16 / DQ4_OUT_F32.  Sums are FP32.
 *
 * A weight is what dq4_int8_correction_prep takes: CB, int8[N][K] row-major, and SCB,
 * FP32[N]; its values are CB[n][k] * SCB[n] / 127.  Rows of activations in 8 bits are the
 * same: codes int8[M][K], scales FP32[M].
 *
 * Workspaces: device memory, 256-byte aligned, of at least the bytes that the function beside
 * the entry point gives (-DQ4_ERR_DEVICE if no device answers), the quantizer's zero before its
 * first use (the others hold anything); a completed call leaves a workspace ready for later calls
 * of the same entry point, of any shape that it is large enough for, in the same stream (not for
 * concurrent calls or replays of captured ones).
 *
 * `bad` is an optional device int (NULL to skip) that counts what a call could not do, as each
 * entry point says, and waits inside a kernel that ran out (never expected; results of that call
 * are not to be used); it stays 0 for valid inputs.
 */
#ifndef DQ4_INT8_H
#define DQ4_INT8_H

#include <stdint.h>

#include "dq4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows of X in 8 bits, each by its largest value:
 *   scale = max |x| over the row's values with |x| < threshold (all of them if threshold
 *           is 0); 0 if that is below 2^-100, and NaN, with codes of 0, if a value is NaN or,
 *           without a threshold, infinite
 *   code  = RN32(x * RN32(127 / scale)) rounded to the nearest integer (ties to even), within
 *           -127 .. 127; 0 where the scale is 0
 * A column with some |x| >= threshold is an outlier.  The first max_cols of them (by index)
 * keep their values: their codes are 0 in every row, and
 *   cols      int64[max_cols]: their indices, ascending, -1 in the rest
 *   outliers  `dtype`[M][max_cols]: their values bit for bit, 0 in the rest
 *   count     int32[1]: the outlier columns found, max_cols or not
 * Outlier columns past max_cols keep their codes, where larger values stand at +-127.
 *   X         `dtype` (FP16 or BF16) [M][K], rows row_stride elements apart, a row's values
 *             contiguous
 *   codes     int8[M][K], scales FP32[M]
 * threshold == 0: cols, outliers, count and workspace are not used (NULL).  threshold < 0
 * or NaN, max_cols outside 1 .. 128, M or K < 0: DQ4_ERR_N.
 * Fastest where K and row_stride (of several rows) are multiples of 8, X 16-byte and codes 8-byte
 * aligned.
 */
int dq4_int8_quantize(const void* X, int64_t row_stride, int32_t dtype, int64_t M, int64_t K,
                      float threshold, int8_t* codes, float* scales, int64_t* cols,
                      int32_t max_cols, void* outliers, int32_t* count, void* workspace,
                      int64_t workspace_bytes, void* stream);
int64_t dq4_int8_quantize_workspace_bytes(int64_t K);

/*
 * The product of rows in 8 bits with a weight in 8 bits:
 *   Y[m][n] = scales[m] SCB[n] / 127^2 * sum_k codes[m][k] CB[n][k]
 *           + SCB[n] / 127 * sum_l outliers[m][l] CB[n][cols[l]]  +  bias[n]
 *   cols      int64[L], outliers `outlier_dtype` (FP16 or BF16) [M][L]: columns in 16 bits, as
 *             dq4_int8_quantize gives them (L 0 .. 128; L == 0: none).  Indices ascend, -1
 *             stands for none; one outside [0, K), or not above all before it, is not used and
 *             counted into bad, but for -1.  The codes of a column that is used are not.
 *   bias      `out_dtype`[N] or NULL
 *   Y         `out_dtype` (FP16, BF16 or FP32) [M][N], row-major
 * The sum over codes is exact while it and its parts stay below 2^24 (always up to K = 1040),
 * beyond that, and together with outliers, rounded as FP32 sums are.  In products of many rows an
 * outlier is held to 2^-22 of it, or 2^-25 of the larger of scales[m] / 127 and 2^-14 of the
 * row's largest outlier, and codes beside one above 2^32 scales[m] to 2^-39 of it; products of few
 * rows hold both to FP32.  A row whose scale is NaN, or with an outlier that is not finite, is NaN.
 * K % 16 == 0, codes and CB 16-byte aligned, M, N, K < 2^31, M * K and N * K < 2^47.
 */
int dq4_int8_linear(const int8_t* codes, const float* scales, const int8_t* CB, const float* SCB,
                    int64_t M, int64_t N, int64_t K, const int64_t* cols, int32_t L,
                    const void* outliers, int32_t outlier_dtype, const void* bias,
                    int32_t out_dtype, void* Y, void* workspace, int64_t workspace_bytes,
                    int* bad, void* stream);
int64_t dq4_int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t L);

/*
 * The gradient of the product's input (the rounding to codes taken as the identity):
 *   dX[m][k] = sum_n dY[m][n] W[n][k],
 *   W[n][k]  = RN16( RN32( RN32(CB[n][k] * SCB[n]) * RN32(1/127) ) ) in dY's type
 *   dY        `dtype` (FP16 or BF16) [M][N], dX `dtype` [M][K], both row-major
 * N % 8 == 0, K % 16 == 0, dY and CB 16-byte aligned; limits as for dq4_int8_linear.
 */
int dq4_int8_linear_backward(const void* dY, int32_t dtype, const int8_t* CB, const float* SCB,
                             int64_t M, int64_t N, int64_t K, void* dX, void* workspace,
                             int64_t workspace_bytes, int* bad, void* stream);
int64_t dq4_int8_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * A mixture-of-experts layer for few tokens:
 *   ids[t]      the top_k experts with the largest logits of token t, in falling order, the
 *               lower index first where they are equal (a NaN counts as -infinity here)
 *   weights[t]  softmax of the logits at those, over all experts, or over the chosen ones if
 *               renormalize; 0 in a row whose logits are all -infinity
 *   Y[t]        sum over j of weights[t][j] * W2[e] (silu(Wg[e] x) * (Wu[e] x)), e = ids[t][j],
 *               x = X[t]; a weight of 0 adds nothing
 *   X           `dtype` (FP16 or BF16) [T][H], rows contiguous, row_stride elements apart
 *   logits      FP32[T][E]
 *   W1, S1      int8[E][2 I][H], FP32[E][2 I]: the rows of Wg, then those of Wu
 *   W2, S2      int8[E][H][I], FP32[E][H]
 *   ids         int32[T][top_k] and weights FP32[T][top_k]: outputs
 *   Y           `dtype`[T][H], contiguous
 * Activations are FP16 in the products, a power of two for each row keeping them in its range
 * (BF16 rows lose nothing down to 2^-31 of their largest value); the inner values are held in
 * two terms of 11 bits: to 2^-22 of them, or 2^-39 of the largest of their row.
 * T 0 .. 256, E 1 .. 1024, top_k 1 .. min(E, 16), H 16 .. 32768 and I 16 .. 2^20, both multiples
 * of 16, E * I * H < 2^47 (H and I may be 0 without tokens); weights 16-byte aligned, X 16-byte
 * aligned, with row_stride % 8 == 0 where there are several tokens.
 */
int dq4_int8_moe(const void* X, int64_t row_stride, int32_t dtype, int64_t T, int64_t H, int64_t I,
                 int64_t E, const float* logits, int32_t top_k, int32_t renormalize,
                 const int8_t* W1, const float* S1, const int8_t* W2, const float* S2,
                 int32_t* ids, float* weights, void* Y, void* workspace,
                 int64_t workspace_bytes, int* bad, void* stream);
int64_t dq4_int8_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int32_t top_k);

#ifdef __cplusplus
}
#endif

#endif /* DQ4_INT8_H */
