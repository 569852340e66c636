/*
 * gq_g4.h -- C ABI of the products with 4-bit weights and group scales
 * (gfx950); part of libgq.so, next to gq.h, whose types, status codes and
 * conventions it uses (device pointers owned by the caller and 16-byte
 * aligned, asynchronous calls, validation on the host before any HIP call,
 * nothing launched and nothing written on an error).
 *
 * Weights.  W is [N][K / 2] bytes, rows back to back: input 2 i of a row is the
 * low, input 2 i + 1 the high nibble of its byte i.  Each group of `group`
 * inputs of a row (32, 64 or 128; the last may be shorter) has a scale, bf16 or
 * fp16, in scales [N][ceil(K / group)], and a zero point, a byte of zeros
 * [N][ceil(K / group)] (0..15, the upper four bits are ignored); zeros may be
 * NULL, every zero point is then 8:
 *   w(n, k) = scales[n][k / group] * (q(n, k) - zeros[n][k / group]).
 *
 * Sizes.  K is a multiple of 32 (rows of W start 16-byte aligned) and at most
 * 4,194,304, N at most 268,435,200, rows (M) at most 2,147,483,392, an operand
 * at most 2^40 elements (GQ_ERR_SHAPE beyond).
 *
 * Experts.  The products of many rows take one matrix (offsets == NULL,
 * n_experts == 1), or n_experts <= 4096 of them and rows sorted by expert:
 * offsets (int32 [n_experts + 1], device, as gq_expert_sort writes them) says
 * that the rows [offsets[e], offsets[e + 1]) belong to expert e, with W
 * [n_experts][N][K / 2], scales and zeros [n_experts][N][ceil(K / group)].  Rows
 * outside [offsets[0], offsets[n_experts]) belong to none: their results are
 * left as they were.  offsets must not decrease and lie in 0..M; others give
 * wrong values but no access out of bounds.
 *
 * Range.  A sum over a group is formed before its scale meets it; the
 * accuracies below hold for fp32 and bf16 inputs that are zero or from 2^-94 up
 * to below 2^112 and fp16 ones of any size, for finite scales of any size, and
 * where sums and results are normal numbers of their type.  A NaN or infinite
 * input or scale makes the outputs that read it NaN or infinite; nothing else is
 * affected by it.
 */
#ifndef GQ_G4_H
#define GQ_G4_H

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Decode product: y[b][n] = sum_k w(n, k) x[b][k] for 1 <= batch <= 16 vectors
 * (GQ_ERR_UNSUPPORTED above).  x: [batch][K], y: [batch][N], each of GQ_F32,
 * GQ_BF16 or GQ_F16.  N == 0 is a no-op; K == 0 writes zeros.
 * Accuracy: q - z and x enter exactly (fp32 vectors, from two on, as three bf16
 * parts), products are exact and sums fp32: within (K / 32 + 2 group + 48) *
 * 2^-23 times sum |w x|, then y_dtype's rounding.  Each vector's result does not
 * depend on the other vectors' values. */
gq_status gq_g4_matvec(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group,
                       int64_t N, int64_t K, const void* x, gq_dtype x_dtype, int32_t batch, void* y,
                       gq_dtype y_dtype, hipStream_t stream);

/* Product of many rows: Y[m][n] = sum_k w(n, k) X[m][k], with offsets by the
 * weights of row m's expert.  X: [M][ldx] of x_dtype (GQ_BF16 or GQ_F16; rows
 * start 16-byte aligned: ldx a multiple of 8, at most 4,194,304), Y: [M][ldy] of
 * y_dtype (GQ_F32 or x_dtype), any ldy >= N.  M == 0 or N == 0 is a no-op; K == 0
 * writes zeros.  Columns past N are not touched.
 * Accuracy.  GQ_F32: as gq_g4_matvec.  Y of X's type: that, or each weight
 * rounded to that type first (by the number of rows), i.e. within half its eps
 * (bf16 2^-8, fp16 2^-11) times sum |w x| more, and 2^-25 |x| where a weight is
 * below fp16's normal numbers, 2^-125 |x| where one is below 2^-117 in bf16;
 * weights of 65520 and more are infinite then in fp16.  Who needs the weights as
 * they are whatever the number of rows takes GQ_F32 results. */
gq_status gq_g4_matmul(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group,
                       int64_t N, int64_t K, const void* X, gq_dtype x_dtype, int64_t M, int64_t ldx, void* Y,
                       gq_dtype y_dtype, int64_t ldy, int32_t n_experts, const int32_t* offsets,
                       hipStream_t stream);

/* Gradient of gq_g4_matmul with respect to X (the weights are constants):
 * dX[m][k] = sum_n w(n, k) dY[m][n].  dY: [M][lddy], dX: [M][lddx] of dtype
 * (GQ_BF16 or GQ_F16), any lddy >= N, lddx >= K.  M == 0 or K == 0 is a no-op;
 * N == 0 writes zeros (with offsets: to the rows of the experts).  Accuracy: each
 * weight is rounded to dtype (see gq_g4_matmul), sums are fp32 (within (N / 32 +
 * 64) * 2^-23 times sum |w dY|), then dtype's rounding. */
gq_status gq_g4_matmul_dx(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group,
                          int64_t N, int64_t K, const void* dY, gq_dtype dtype, int64_t M, int64_t lddy, void* dX,
                          int64_t lddx, int32_t n_experts, const int32_t* offsets, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_G4_H */
