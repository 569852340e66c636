// gq_expert_abi.cpp -- the extern "C" boundary of gq_expert.h: argument
// validation (before any HIP call) and dispatch to the kernel launchers.
#include "../../include/gq_expert.h"

#include <hip/hip_runtime.h>

#include "gq_expert_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gq_status from_hip(hipError_t e) { return e == hipSuccess ? GQ_OK : GQ_ERR_LAUNCH; }

// Largest element count of any operand, most slots and longest row.
constexpr int64_t MAX_ELEMS = (int64_t)1 << 40;
constexpr int64_t MAX_SLOTS = (int64_t)1 << 20;
constexpr int64_t MAX_D = ((int64_t)1 << 28) - 256;

// rows x stride elements within MAX_ELEMS (both already known to be >= 0)
bool fits(int64_t rows, int64_t stride) { return rows == 0 || stride <= MAX_ELEMS / rows; }

bool is_dtype(gq_dtype t) { return t == GQ_F32 || t == GQ_BF16 || t == GQ_F16; }

bool bad_slots(int32_t n_tokens, int32_t top_k) {
    return n_tokens < 0 || top_k < 1 || (int64_t)n_tokens * top_k > MAX_SLOTS;
}

}  // namespace

extern "C" {

gq_status gq_expert_sort(const int32_t* ids, int32_t n_tokens, int32_t top_k, int32_t n_experts, int32_t* offsets,
                         int32_t* place, hipStream_t stream) {
    if (bad_slots(n_tokens, top_k) || n_experts < 1) return GQ_ERR_SHAPE;
    if (n_experts > 4096) return GQ_ERR_UNSUPPORTED;
    if (!offsets || (n_tokens > 0 && (!ids || !place))) return GQ_ERR_NULL;
    if (!aligned16(offsets) || (n_tokens > 0 && (!aligned16(ids) || !aligned16(place)))) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_expert_sort(ids, n_tokens, top_k, n_experts, offsets, place, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_expert_gather(const void* x, gq_dtype dtype, int32_t n_tokens, int32_t top_k, int64_t D, int64_t ldx,
                           const int32_t* place, void* xs, int64_t ldxs, hipStream_t stream) {
    if (!is_dtype(dtype)) return GQ_ERR_DTYPE;
    if (bad_slots(n_tokens, top_k) || D < 0 || D > MAX_D || ldx < D || ldxs < D) return GQ_ERR_SHAPE;
    if (!fits(n_tokens, ldx) || !fits((int64_t)n_tokens * top_k, ldxs)) return GQ_ERR_SHAPE;
    if (n_tokens == 0 || D == 0) return GQ_OK;
    if (!x || !place || !xs) return GQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(place) || !aligned16(xs)) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_expert_gather(x, dtype, n_tokens, top_k, D, ldx, place, xs, ldxs, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_expert_combine(const void* ys, gq_dtype dtype, int32_t n_tokens, int32_t top_k, int64_t D, int64_t ldys,
                            const int32_t* place, const float* weights, void* y, gq_dtype y_dtype, int64_t ldy,
                            hipStream_t stream) {
    if (!is_dtype(dtype) || (y_dtype != GQ_F32 && y_dtype != dtype)) return GQ_ERR_DTYPE;
    if (bad_slots(n_tokens, top_k) || D < 0 || D > MAX_D || ldys < D || ldy < D) return GQ_ERR_SHAPE;
    if (!fits((int64_t)n_tokens * top_k, ldys) || !fits(n_tokens, ldy)) return GQ_ERR_SHAPE;
    if (n_tokens == 0 || D == 0) return GQ_OK;
    if (!ys || !place || !y) return GQ_ERR_NULL;
    if (!aligned16(ys) || !aligned16(place) || !aligned16(y) || (weights && !aligned16(weights))) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_expert_combine(ys, dtype, n_tokens, top_k, D, ldys, place, weights, y, y_dtype, ldy,
                                           stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_expert_combine_grad(const void* dy, gq_dtype dtype, int32_t n_tokens, int32_t top_k, int64_t D,
                                 int64_t lddy, const void* ys, int64_t ldys, const int32_t* place,
                                 const float* weights, void* dys, int64_t lddys, float* dweights,
                                 hipStream_t stream) {
    if (!is_dtype(dtype)) return GQ_ERR_DTYPE;
    const int64_t slots = (int64_t)n_tokens * top_k;
    if (bad_slots(n_tokens, top_k) || D < 0 || D > MAX_D || lddy < D || !fits(n_tokens, lddy)) return GQ_ERR_SHAPE;
    if (dweights && (ldys < D || !fits(slots, ldys))) return GQ_ERR_SHAPE;
    if (dys && (lddys < D || !fits(slots, lddys))) return GQ_ERR_SHAPE;
    if (n_tokens == 0 || (!dys && !dweights) || (D == 0 && !dweights)) return GQ_OK;
    if (!place || (D > 0 && (!dy || (dweights && !ys)))) return GQ_ERR_NULL;
    if (!aligned16(place) || (D > 0 && (!aligned16(dy) || (dweights && !aligned16(ys)))) || (dys && !aligned16(dys)) ||
        (weights && !aligned16(weights)) || (dweights && !aligned16(dweights)))
        return GQ_ERR_ALIGN;
    if (dys && dweights && dys == ys && lddys != ldys) return GQ_ERR_SHAPE;
    try {
        return from_hip(gqk_expert_combine_grad(dy, dtype, n_tokens, top_k, D, lddy, ys, ldys, place, weights, dys,
                                                lddys, dweights, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

}  // extern "C"
