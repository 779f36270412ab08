/*
 * sgemm_experts.h -- products grouped by expert, and 4-bit microscaled
 * (MXFP4) operands (GB300, sm_103a).  Companion of sgemm.h: same status codes,
 * streams, error behaviour and scratch pool.
 *
 * Types.  A `type` argument names the element type of the operands in HBM.
 * Every product accumulates in float32 and rounds once, to nearest even, to
 * the output's type.
 *
 * Groups.  A token array holds T rows sorted by expert.  `offsets` is a DEVICE
 * array of E + 1 ints: expert e owns rows offsets[e] .. offsets[e + 1] - 1.
 * The host never reads it, so nothing waits for the GPU.  The kernels take
 * every entry clamped to [0, T] and as the running maximum of the entries so
 * far, so that no value in it can make them leave the arrays: a decreasing
 * entry makes an empty group.  Rows before offsets[0] and from offsets[E] on
 * belong to no expert.
 *
 * Memory.  All pointers are DEVICE pointers owned by the caller and aligned
 * to their element type; leading dimensions and strides are in elements.
 * Outputs must not overlap inputs.  Row padding is never written and never
 * reaches a result.  It may be read, and so may what lies around an operand,
 * but only bytes that share an aligned 16 with one of its elements.
 * Entry points that may allocate device memory from the library's
 * stream-ordered pool (see sgemm.h), freed in stream order at the end of the
 * call, and those that never do:
 *   EXPERTS-ALLOCATING: sgemm_grouped sgemm_grouped_wgrad
 *   EXPERTS-NON-ALLOCATING: sgemm_mxfp4_quantize sgemm_mxfp4_dequantize sgemm_mxfp4 sgemm_mxfp4_grouped
 * (16-bit operands whose base or rows are off the 16-byte grid are copied into
 * pitched rows, float32 operands into three bf16 parts, 6 bytes an element,
 * but for forward products of few rows an expert.)
 */
#ifndef GB300_SGEMM_EXPERTS_H
#define GB300_SGEMM_EXPERTS_H

#include <stdint.h>

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { SGEMM_TYPE_F32 = 0, SGEMM_TYPE_BF16 = 1, SGEMM_TYPE_F16 = 2 };

/*
 * sgemm_grouped -- rows times their expert's weights
 *
 *     Y[t, :] = X[t, :] op(W_e)    for offsets[e] <= t < offsets[e + 1],
 *     Y[t, :] = 0                  for rows that belong to no expert.
 *
 *   type       of X, W and Y
 *   transw     0: op(W_e) = W_e, stored K x N (ldw >= N);
 *              1: op(W_e) = W_e^T, W_e stored N x K (ldw >= K).  With the
 *              weights of a forward call and transw inverted this is the
 *              gradient of its rows: dX = dY op(W_e)^T
 *   T, E, N, K rows, experts, row widths of Y and X (all >= 0)
 *   X, ldx     T x K
 *   W, ldw, stride_w   E matrices, stride_w elements apart
 *   offsets    E + 1 ints on the device (see "Groups" above)
 *   Y, ldy     T x N, overwritten
 * Accuracy: float32 operands as the other entries, |Y - exact| <= 5e-5 *
 * sum_k |X_tk||op(W)_kn|; bf16 and f16 operands that bound plus one rounding
 * to the type.  It holds whatever the operands' signs and magnitudes for
 * contractions up to 2^17 (what goes into one accumulator is limited); every
 * further 2^10 may add 2^-22 times the sum.  (float32 operands that go to the
 * tensor cores as parts are taken to a multiple of 2^-133, which those below
 * 2^-118 in magnitude notice: 5e-5 holds from about 2^-122 on.)
 * A non-finite operand reaches only its own row (X) or its own column of its
 * expert's rows (W); where it reaches, float32 results are not finite, but may
 * be NaN where the exact result is an infinity.
 */
int sgemm_grouped(int type, int transw, int T, int E, int N, int K,
                  const void* X, int64_t ldx,
                  const void* W, int64_t ldw, int64_t stride_w,
                  const int* offsets,
                  void* Y, int64_t ldy,
                  void* stream);

/*
 * sgemm_grouped_wgrad -- the gradient of every expert's weights
 *
 *     dW_e = X_e^T dY_e = sum over the expert's rows t of X[t, :]^T dY[t, :]
 *
 * (K x N; zeros for an expert without rows).  For weights stored N x K
 * (transw = 1 in the forward call) pass dY as X and X as dY.
 *   type       of X and dY
 *   out_type   of dW: `type` or SGEMM_TYPE_F32
 *   X, ldx     T x K;   dY, lddy   T x N
 *   dW, lddw, stride_dw   E matrices, overwritten
 * Accuracy as sgemm_grouped; the contraction is an expert's rows.
 */
int sgemm_grouped_wgrad(int type, int out_type, int T, int E, int K, int N,
                        const void* X, int64_t ldx,
                        const void* dY, int64_t lddy,
                        const int* offsets,
                        void* dW, int64_t lddw, int64_t stride_dw,
                        void* stream);

/*
 * MXFP4.  A row of K values is held as 4-bit codes with one scale for each
 * block of 32 consecutive columns:
 *     value = e2m1(code) * 2^(scale - 127),
 * e2m1 magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 for codes 0..7, bit 3 the sign.
 *
 * codes: rows of 16 * ceil(K / 32) bytes, the even column in a byte's low
 * four bits; columns past K hold zeros.  16-byte aligned.
 *
 * scales: bytes in blocks of 128 rows x 4 scales, 512 bytes each, in the order
 * in which the tensor cores read them: element (row r, scale b) of a matrix of
 * ceil(R / 128) x ceil(K / 128) blocks is byte
 *     ((r / 128) * ceil(K / 128) + b / 4) * 512 + (r % 32) * 16
 *         + (r % 128 / 32) * 4 + b % 4.
 * 16-byte aligned.  Scales of rows beyond the matrix are present and may hold
 * anything; those of columns beyond it, anything but 255 (the quantiser writes
 * zeros).
 * Rows grouped by expert: every expert's rows begin a new block of 128 (the
 * experts' blocks follow one another, none for an expert without rows), so
 * that T rows take at most (T + 127 min(T, E)) / 128 row blocks.
 */

/*
 * sgemm_mxfp4_quantize -- MXFP4 form of the rows of X
 *
 * For each block, m = its largest magnitude, s = max(floor(log2 m) - 2, -127):
 * scale byte s + 127 (0 for a block of zeros), codes x * 2^-s rounded to
 * nearest, ties to the even code, magnitudes beyond 6 to 6.  A block with an
 * infinity or a NaN gets the scale byte 255, with which all its values stand
 * for NaN, whatever their codes.
 *   type       of X
 *   batch, rows, K   X is `batch` matrices of rows x K, stride_x apart
 *   E, offsets NULL: each matrix has scale blocks of its own.  Otherwise
 *              batch = 1 and the rows are grouped by E experts (scales laid out
 *              as above; rows that belong to no expert get codes, and no
 *              scales)
 *   codes, scales   outputs, batch matrices one after the other
 */
int sgemm_mxfp4_quantize(int type, int batch, int rows, int K,
                         const void* X, int64_t ldx, int64_t stride_x,
                         int E, const int* offsets,
                         uint8_t* codes, uint8_t* scales,
                         void* stream);

/*
 * sgemm_mxfp4_dequantize -- the values that codes and scales stand for, to Y
 * (batch matrices of rows x K of `type`, stride_y apart); E and offsets as
 * given to the quantiser.  Rows that belong to no expert get zeros.  Values
 * are exact in float32 and bf16 up to scale byte 252, the quantiser's largest;
 * above it those beyond the type's range are infinities.
 */
int sgemm_mxfp4_dequantize(int type, int batch, int rows, int K,
                           const uint8_t* codes, const uint8_t* scales,
                           int E, const int* offsets,
                           void* Y, int64_t ldy, int64_t stride_y,
                           void* stream);

/*
 * sgemm_mxfp4 -- C = A B^T of two MXFP4 matrices, A (M x K) and B (N x K), both
 * quantised along K; C (M x N) of out_type.  Products are exact, sums are in
 * float32: |C - exact| <= 5e-5 * sum_k |a||b| plus the rounding to out_type, for
 * contractions up to 2^20 and sums of magnitudes within float32's range; below
 * its normal numbers every 64 of the contraction may add 2^-149.
 */
int sgemm_mxfp4(int out_type, int M, int N, int K,
                const uint8_t* A, const uint8_t* a_scales,
                const uint8_t* B, const uint8_t* b_scales,
                void* C, int64_t ldc,
                void* stream);

/*
 * sgemm_mxfp4_grouped -- Y[t, :] = X[t, :] W_e^T for the rows of each expert,
 * zeros for rows of none: X (T x K) quantised with the same offsets, W E
 * matrices of N x K one after the other, each with scale blocks of its own.
 */
int sgemm_mxfp4_grouped(int out_type, int T, int E, int N, int K,
                        const uint8_t* X, const uint8_t* x_scales,
                        const uint8_t* W, const uint8_t* w_scales,
                        const int* offsets,
                        void* Y, int64_t ldy,
                        void* stream);

#ifdef __cplusplus
}
#endif
#endif
