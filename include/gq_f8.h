/*
 * gq_f8.h -- C ABI of the block-scaled 8-bit products and of the router with
 * scores (gfx950); part of libgq.so, next to gq.h, whose types, status codes
 * and conventions it uses (device pointers owned by the caller and 16-byte
 * aligned, asynchronous calls, validation on the host before any HIP call,
 * nothing launched and nothing written on an error).
 *
 * Weights.  W is [N][K] bytes of e4m3 (1 sign, 4 exponent, 3 mantissa bits,
 * bias 7, largest value 448, S.1111.111 = NaN, no infinity), rows back to
 * back, with one fp32 scale for each block of 128 rows x 128 inputs:
 * wscales [ceil(N / 128)][ceil(K / 128)], weight (n, k) =
 * W[n][k] * wscales[n / 128][k / 128].  Blocks at the right and lower edge
 * may be partial.
 *
 * Activations of the products of two 8-bit operands: e4m3 rows with one fp32
 * scale for each 128 inputs of a row, stored group by group:
 * xscales[k / 128][m] (row stride xs_ld >= M), so that the scales of
 * neighbouring rows are neighbours in memory.  gq_f8_quant and
 * gq_f8_glu_quant write this form.
 *
 * Sizes.  K is a multiple of 16 (rows of bytes start 16-byte aligned) and at
 * most 4,194,304 everywhere, as is the row stride ldx of the products of two
 * 8-bit operands; N at most 268,435,200; rows (M) at most 2,147,483,392; an
 * operand at most 2^40 elements (GQ_ERR_SHAPE beyond).
 *
 * Range.  The sum over a block of 128 inputs is formed before its scales meet
 * it, and the two scales of a product are multiplied first, in fp32.  The
 * accuracies below hold for vectors (gq_f8_matvec) of zeros and values from
 * 2^-94 up to below 2^112, and for pairs of scales whose product is a normal
 * fp32 number; beyond, a result may be an infinity, NaN or zero where the exact
 * one is a number.
 *
 * A NaN weight, activation or scale makes the outputs that read it NaN; nothing
 * else is affected by it.
 */
#ifndef GQ_F8_H
#define GQ_F8_H

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations to 8 bits: for each row m and each group b of 128 inputs (the
 * last may be shorter), with a = max |x[m][k]| over the group,
 *   s = a / 448 in fp32, at least 2^-64; with pow2 != 0 the smallest power of
 *       two >= that;
 *   q[m][k] = the e4m3 value nearest to the fp32 quotient x[m][k] / s (ties to
 *       the even one), scales[b][m] = s.
 * Bit-exact (a zero may have either sign).  A group that holds an infinity or
 * NaN gets s = NaN and q = 0 (every product with it is NaN).
 * x: [M][ldx] of x_dtype (GQ_F32, GQ_BF16, GQ_F16); q: [M][ldq] bytes; scales:
 * [ceil(K / 128)][s_ld] fp32 (s_ld >= M).  Rows of x and q must start at
 * multiples of 16 bytes.  Elements past K or M are not touched. */
gq_status gq_f8_quant(const void* x, gq_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, int32_t pow2, void* q,
                      int64_t ldq, float* scales, int64_t s_ld, hipStream_t stream);

/* The gated unit's elementwise step straight to 8 bits: gq_f8_quant of
 *   h[m][k] = act(g[m][k]) * u[m][k]
 * computed in fp32 and not rounded in between (act as gq_matvec_glu's; h within
 * 2^-20 |h| + 2^-125 |g u|, with the tanh form within 2^-20 (|h| + |g u|)).
 * g, u: [M][ldg], [M][ldu] of dtype (the halves of one gate|up product, or two). */
gq_status gq_f8_glu_quant(const void* g, const void* u, gq_dtype dtype, int64_t M, int64_t K, int64_t ldg,
                          int64_t ldu, gq_act act, int32_t pow2, void* q, int64_t ldq, float* scales, int64_t s_ld,
                          hipStream_t stream);

/* Decode product: y[b][n] = sum_k w[n][k] x[b][k] for 1 <= batch <= 16
 * vectors (GQ_ERR_UNSUPPORTED above).  x: [batch][K] of x_dtype (GQ_F32 or
 * GQ_BF16), not quantised; y: [batch][N] of y_dtype (GQ_F32 or GQ_BF16).
 * N == 0 is a no-op; K == 0 writes zeros.
 * Accuracy: weights and activations enter exactly (fp32 ones, from two vectors
 * on, as three bf16 parts), products are exact and sums fp32: within (K / 128 +
 * 162) * 2^-23 times sum |w x| (fp32 vectors: K / 128 + 418, their parts being
 * three sums), then y_dtype's rounding.  An infinite activation gives NaN or an
 * infinity.  Each vector's result does not depend on the other vectors' values. */
gq_status gq_f8_matvec(const void* W, const float* wscales, int64_t N, int64_t K, const void* x, gq_dtype x_dtype,
                       int32_t batch, void* y, gq_dtype y_dtype, hipStream_t stream);

/* Product of two 8-bit operands: Y[m][n] = sum over groups b of 128 inputs of
 *   xscales[b][m] * wscales[n / 128][b] * sum_{k in b} X[m][k] W[n][k].
 * X: [M][ldx] e4m3 bytes (ldx a multiple of 16), xscales [ceil(K/128)][xs_ld],
 * Y: [M][ldy] of y_dtype (GQ_F32 or GQ_BF16), any ldy >= N.  M == 0 or N == 0
 * is a no-op; K == 0 writes zeros.  Columns past N are not touched.
 * Accuracy.  GQ_F32: the operands are widened to bf16 (exact), sums are fp32:
 * within (K / 128 + 162) * 2^-23 times sum |x w|.  GQ_BF16: the 8-bit matrix
 * instructions run at twice that rate and keep, of every eight products they
 * add, the bits down to 2^-13 of the largest's exponent: within 2^-10 times
 * sum |x w| at worst (e4m3 subnormals counted as 2^-6), about 2^-16 of the
 * result's size on ordinary data; then bf16's rounding. */
gq_status gq_f8_matmul(const void* W, const float* wscales, int64_t N, int64_t K, const void* X,
                       const float* xscales, int64_t M, int64_t ldx, int64_t xs_ld, void* Y, gq_dtype y_dtype,
                       int64_t ldy, hipStream_t stream);

/* Workspace bytes of gq_f8_matmul_id for these sizes (host only): a table of
 * the slots by expert and, for a weighted product, the per-slot outputs. */
gq_status gq_f8_matmul_id_workspace(int32_t n_experts, int32_t n_tokens, int32_t top_k, int64_t N, gq_dtype y_dtype,
                                    int32_t weighted, size_t* bytes);

/* Routed-expert product of two 8-bit operands, from one token to a prompt:
 * for slot (t, j) with e = ids[t][j], gq_f8_matmul's row with the weights
 * experts[e] ([n_experts][N][K] bytes, wscales [n_experts][ceil(N/128)]
 * [ceil(K/128)]).  X: [n_tokens][ldx] (x_per_slot == 0: a token's slots read
 * the token's row) or [n_tokens * top_k][ldx] (x_per_slot == 1), xscales as
 * for gq_f8_matmul with as many rows.
 *   route_w == NULL: Y is [n_tokens][top_k][N] of y_dtype.
 *   route_w != NULL (fp32 [n_tokens][top_k]): Y is [n_tokens][N],
 *     Y[t][n] = sum_j route_w[t][j] * slot[t][j][n], j in increasing order,
 *     in fp32; the slot values are held in y_dtype (with GQ_BF16 each carries
 *     one rounding more than the result's own).
 * An expert's weights are read once for all of its slots that share a tile.
 * ids: int32 [n_tokens][top_k] (device).  ids may be NULL: the table in ws,
 * left by the previous call with the same ws, n_experts, n_tokens, top_k and
 * ids, is used (its fields are clamped: a workspace that holds no table gives
 * wrong values but no access out of bounds).  An id outside [0, n_experts)
 * makes its slot contribute zero (its row of an unweighted Y is zeroed; with
 * ids == NULL left as it was) and is counted (gq_f8_matmul_id_check).
 * n_experts <= 4096, 1 <= top_k <= n_experts, n_tokens * top_k <= 1,048,576.
 * ws: gq_f8_matmul_id_workspace bytes, no initialisation needed; calls that
 * share it must be ordered.  n_tokens == 0 or N == 0 is a no-op; K == 0 gives
 * zeros.  Accuracy of a slot as gq_f8_matmul. */
gq_status gq_f8_matmul_id(const void* experts, const float* wscales, int32_t n_experts, int64_t N, int64_t K,
                          const int32_t* ids, int32_t n_tokens, int32_t top_k, const void* X, const float* xscales,
                          int64_t ldx, int64_t xs_ld, int32_t x_per_slot, const float* route_w, void* Y,
                          gq_dtype y_dtype, void* ws, size_t ws_bytes, hipStream_t stream);

/* Waits for `stream`, then reports how many ids of the last gq_f8_matmul_id
 * call given ids that used `ws` were outside [0, n_experts). */
gq_status gq_f8_matmul_id_check(const void* ws, hipStream_t stream, int32_t* n_bad_ids);

/* Scores of gq_route_scored and the value by which it ranks groups. */
typedef enum { GQ_SCORE_SOFTMAX = 0, GQ_SCORE_SIGMOID = 1 } gq_score;
typedef enum { GQ_GROUP_MAX = 0, GQ_GROUP_TOP2 = 1 } gq_group_rank;

/* Expert routing by scores.  For each token t with logits l[e] (GQ_F32 or
 * GQ_BF16, [n_tokens][n_experts]):
 *   s[e] = 1 / (1 + exp(-l[e])), or the softmax of l over all experts (0 for
 *          every expert when all logits are -inf);
 *   c[e] = s[e] + bias[e] (bias: fp32 [n_experts] or NULL; it takes part in
 *          the choice only);
 *   the experts form n_groups runs of n_experts / n_groups; a group's value is
 *   its largest c or the sum of its two largest (c alone in a group of one);
 *   the top_groups groups of the largest value stay;
 *   ids[t]: of their experts the top_k of the largest c, in decreasing order;
 *   weights[t][j] = scale * s[ids[t][j]], with renorm != 0 divided by the sum
 *   of the chosen s (0 when that sum is 0).
 * Equal values: the lower index first.  s, c and group values are computed in
 * 64 bits, so the choice is exact up to scores that differ by less than about
 * 2^-50; a c or group value that is NaN counts as -inf.  weights are fp32
 * (one rounding of a 64-bit value).  A bias of -inf keeps an expert out as
 * long as others are left.
 * n_experts <= 4096, top_k <= 64, n_groups <= 64 (GQ_ERR_UNSUPPORTED beyond);
 * n_tokens <= 33,554,432;
 * n_groups divides n_experts, 1 <= top_groups <= n_groups, 1 <= top_k <=
 * top_groups * n_experts / n_groups (GQ_ERR_SHAPE otherwise).  n_tokens == 0
 * is a no-op.  ids and weights feed gq_matvec_id and gq_f8_matmul_id. */
gq_status gq_route_scored(const void* logits, gq_dtype logits_dtype, int32_t n_tokens, int32_t n_experts,
                          int32_t top_k, gq_score score, const float* bias, int32_t n_groups, int32_t top_groups,
                          gq_group_rank group_rank, int32_t renorm, float scale, int32_t* ids, float* weights,
                          hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_F8_H */
