/*
 * gq_expert.h -- C ABI of tokens sorted by expert and back (gfx950); part of
 * libgq.so, next to gq.h, whose types, status codes and conventions it uses
 * (device pointers owned by the caller and 16-byte aligned, asynchronous calls,
 * validation on the host before any HIP call, nothing launched and nothing
 * written on an error).
 *
 * A routing gives each of n_tokens tokens top_k slots (ids, as gq_route_topk
 * and gq_route_scored write them).  Sorted, the slots of expert 0 come first,
 * then those of expert 1, ..., the slots of one expert in the order of the
 * tokens; slot (t, j) has the place place[t][j] among them.  Per-slot rows at
 * those places are what gq_g4_matmul and gq_g4_matmul_dx take.
 *
 * Rows: n_tokens * top_k of them, D elements of GQ_F32, GQ_BF16 or GQ_F16, any
 * stride >= D and any D (rows whose stride is a multiple of 16 bytes are the
 * fastest).  n_tokens * top_k <= 1,048,576 slots, D <= 268,435,200, an operand
 * at most 2^40 elements (GQ_ERR_SHAPE beyond).  A place outside
 * [0, n_tokens * top_k) stands for a slot without a row; no two slots may have
 * the same one (gq_expert_sort gives none twice; a result row of two slots is
 * one of theirs, piece by piece).  Results lie apart from the inputs and from
 * each other, but for dys, which may be ys.  Every result is the
 * same each time: sums have one order, nothing is added atomically to an output.
 */
#ifndef GQ_EXPERT_H
#define GQ_EXPERT_H

#include "gq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* place[t][j] = the slots of experts below ids[t][j] + the earlier slots of the
 * same expert (both in row-major order of [n_tokens][top_k]); offsets[e] = the
 * slots of experts below e, offsets[n_experts] = all valid slots.  An id
 * outside [0, n_experts) gets place -1 and is not counted.  Any number of a
 * token's slots may have the same expert.
 * ids, place: int32 [n_tokens][top_k]; offsets: int32 [n_experts + 1].
 * 1 <= n_experts <= 4096 (GQ_ERR_UNSUPPORTED above), top_k >= 1.  n_tokens ==
 * 0 writes zeros to offsets. */
gq_status gq_expert_sort(const int32_t* ids, int32_t n_tokens, int32_t top_k, int32_t n_experts, int32_t* offsets,
                         int32_t* place, hipStream_t stream);

/* xs[place[t][j]] = x[t] for every slot with a place (bit for bit); the other
 * rows of xs are left as they were.  x: [n_tokens][ldx], xs: [n_tokens * top_k]
 * [ldxs] of dtype.  n_tokens == 0 or D == 0 is a no-op.  Its gradient is
 * gq_expert_combine with weights NULL. */
gq_status gq_expert_gather(const void* x, gq_dtype dtype, int32_t n_tokens, int32_t top_k, int64_t D, int64_t ldx,
                           const int32_t* place, void* xs, int64_t ldxs, hipStream_t stream);

/* y[t] = sum over the token's slots with a place, in the order of j, of
 * weights[t][j] * ys[place[t][j]], in fp32 (one rounding a slot), rounded once
 * to y_dtype; zeros for a token without any.  weights: fp32 [n_tokens][top_k],
 * or NULL (every weight 1).  ys: [n_tokens * top_k][ldys] of dtype, y:
 * [n_tokens][ldy] of y_dtype (GQ_F32 or dtype).  n_tokens == 0 or D == 0 is a
 * no-op. */
gq_status gq_expert_combine(const void* ys, gq_dtype dtype, int32_t n_tokens, int32_t top_k, int64_t D, int64_t ldys,
                            const int32_t* place, const float* weights, void* y, gq_dtype y_dtype, int64_t ldy,
                            hipStream_t stream);

/* Gradient of gq_expert_combine: for every slot with a place p = place[t][j],
 *   dys[p] = weights[t][j] * dy[t] (rounded once to dtype; weights NULL: dy[t]),
 *   dweights[t][j] = sum_d dy[t][d] * ys[p][d] (fp32 sums, within (D / 256 + 12)
 *   * 2^-23 times the sum of the absolute values),
 * and dweights = 0 for a slot without a place; the other rows of dys are left
 * as they were.  Either result may be NULL (ys too where dweights is).  dy:
 * [n_tokens][lddy], ys: [n_tokens * top_k][ldys], dys: [..][lddys] of dtype;
 * dys may be ys (the same pointer and stride).  n_tokens == 0 is a no-op; D ==
 * 0 gives dweights = 0. */
gq_status gq_expert_combine_grad(const void* dy, gq_dtype dtype, int32_t n_tokens, int32_t top_k, int64_t D,
                                 int64_t lddy, const void* ys, int64_t ldys, const int32_t* place,
                                 const float* weights, void* dys, int64_t lddys, float* dweights,
                                 hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_EXPERT_H */
