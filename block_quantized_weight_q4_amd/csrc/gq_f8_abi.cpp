// gq_f8_abi.cpp -- the extern "C" boundary of gq_f8.h: argument validation
// (before any HIP call) and dispatch to the kernel launchers.
#include "../../include/gq_f8.h"

#include <hip/hip_runtime.h>

#include "gq_f8_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gq_status from_hip(hipError_t e) { return e == hipSuccess ? GQ_OK : GQ_ERR_LAUNCH; }

// Largest element count of any operand, and the longest row (as in gq_abi.cpp).
constexpr int64_t MAX_ELEMS = (int64_t)1 << 40;
constexpr int64_t MAX_K = (int64_t)1 << 22;
constexpr int64_t MAX_SLOTS = (int64_t)1 << 20;

// rows x stride elements within MAX_ELEMS (both already known to be >= 0)
bool fits(int64_t rows, int64_t stride) { return rows == 0 || stride <= MAX_ELEMS / rows; }

int64_t blocks(int64_t n) { return (n + 127) / 128; }

bool bad_k(int64_t K) { return K < 0 || K % 16 != 0 || K > MAX_K; }

// M <= 2^31 - 256: tiles are counted in 32 bits; N and a call's tokens to route:
// a launch has at most 2^32 threads
constexpr int64_t MAX_ROWS = ((int64_t)1 << 31) - 256;
constexpr int64_t MAX_N = ((int64_t)1 << 28) - 256;
constexpr int64_t MAX_TOKENS = (int64_t)1 << 25;

gq_status check_quant(gq_dtype dtype, int64_t M, int64_t K, int64_t ld0, int64_t ld1, int64_t ldq, int64_t s_ld) {
    if (dtype != GQ_F32 && dtype != GQ_BF16 && dtype != GQ_F16) return GQ_ERR_DTYPE;
    if (M < 0 || M > MAX_ROWS || bad_k(K) || ld0 < K || ld1 < K || ldq < K || s_ld < M) return GQ_ERR_SHAPE;
    if (!fits(M, ld0) || !fits(M, ld1) || !fits(M, ldq) || !fits(blocks(K), s_ld)) return GQ_ERR_SHAPE;
    return GQ_OK;
}

// elements per 16 bytes: a stride of rows that must start 16-byte aligned is a multiple of this
int64_t per16(gq_dtype t) { return t == GQ_F32 ? 4 : 8; }

}  // namespace

extern "C" {

gq_status gq_f8_quant(const void* x, gq_dtype x_dtype, int64_t M, int64_t K, int64_t ldx, int32_t pow2, void* q,
                      int64_t ldq, float* scales, int64_t s_ld, hipStream_t stream) {
    const gq_status st = check_quant(x_dtype, M, K, ldx, ldx, ldq, s_ld);
    if (st != GQ_OK) return st;
    if (M == 0 || K == 0) return GQ_OK;
    if (!x || !q || !scales) return GQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(scales)) return GQ_ERR_ALIGN;
    if (M > 1 && (ldx % per16(x_dtype) != 0 || ldq % 16 != 0)) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_f8_quant(x, x_dtype, M, K, ldx, pow2 != 0, static_cast<uint8_t*>(q), ldq, scales, s_ld,
                                     stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_f8_glu_quant(const void* g, const void* u, gq_dtype dtype, int64_t M, int64_t K, int64_t ldg,
                          int64_t ldu, gq_act act, int32_t pow2, void* q, int64_t ldq, float* scales, int64_t s_ld,
                          hipStream_t stream) {
    const gq_status st = check_quant(dtype, M, K, ldg, ldu, ldq, s_ld);
    if (st != GQ_OK) return st;
    if (act != GQ_ACT_SILU && act != GQ_ACT_GELU_TANH) return GQ_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return GQ_OK;
    if (!g || !u || !q || !scales) return GQ_ERR_NULL;
    if (!aligned16(g) || !aligned16(u) || !aligned16(q) || !aligned16(scales)) return GQ_ERR_ALIGN;
    if (M > 1 && (ldg % per16(dtype) != 0 || ldu % per16(dtype) != 0 || ldq % 16 != 0)) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_f8_glu_quant(g, u, dtype, M, K, ldg, ldu, act, pow2 != 0, static_cast<uint8_t*>(q), ldq,
                                         scales, s_ld, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_f8_matvec(const void* W, const float* wscales, int64_t N, int64_t K, const void* x, gq_dtype x_dtype,
                       int32_t batch, void* y, gq_dtype y_dtype, hipStream_t stream) {
    if (x_dtype != GQ_F32 && x_dtype != GQ_BF16) return GQ_ERR_DTYPE;
    if (y_dtype != GQ_F32 && y_dtype != GQ_BF16) return GQ_ERR_DTYPE;
    if (N < 0 || N > MAX_N || bad_k(K) || !fits(N, K) || batch < 1) return GQ_ERR_SHAPE;
    if (batch > 16) return GQ_ERR_UNSUPPORTED;
    if (N == 0) return GQ_OK;
    if (!y || (K > 0 && (!W || !wscales || !x))) return GQ_ERR_NULL;
    if (!aligned16(y) || (K > 0 && (!aligned16(W) || !aligned16(wscales) || !aligned16(x)))) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_f8_matvec(static_cast<const uint8_t*>(W), wscales, N, K, x, x_dtype, batch, y, y_dtype,
                                      stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_f8_matmul(const void* W, const float* wscales, int64_t N, int64_t K, const void* X,
                       const float* xscales, int64_t M, int64_t ldx, int64_t xs_ld, void* Y, gq_dtype y_dtype,
                       int64_t ldy, hipStream_t stream) {
    if (y_dtype != GQ_F32 && y_dtype != GQ_BF16) return GQ_ERR_DTYPE;
    if (N < 0 || M < 0 || N > MAX_N || M > MAX_ROWS || bad_k(K)) return GQ_ERR_SHAPE;
    if (ldx < K || ldx > MAX_K || xs_ld < M || ldy < N) return GQ_ERR_SHAPE;
    if (!fits(N, K) || !fits(M, ldx) || !fits(M, ldy) || !fits(blocks(K), xs_ld)) return GQ_ERR_SHAPE;
    if (M == 0 || N == 0) return GQ_OK;
    if (!Y || (K > 0 && (!W || !wscales || !X || !xscales))) return GQ_ERR_NULL;
    if (!aligned16(Y) || (K > 0 && (!aligned16(W) || !aligned16(wscales) || !aligned16(X) || !aligned16(xscales))))
        return GQ_ERR_ALIGN;
    if (K > 0 && M > 1 && ldx % 16 != 0) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_f8_matmul(static_cast<const uint8_t*>(W), wscales, N, K, static_cast<const uint8_t*>(X),
                                      xscales, M, ldx, xs_ld, Y, y_dtype, ldy, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_f8_matmul_id_workspace(int32_t n_experts, int32_t n_tokens, int32_t top_k, int64_t N, gq_dtype y_dtype,
                                    int32_t weighted, size_t* bytes) {
    if (!bytes) return GQ_ERR_NULL;
    if (y_dtype != GQ_F32 && y_dtype != GQ_BF16) return GQ_ERR_DTYPE;
    if (n_experts < 1 || n_tokens < 0 || top_k < 1 || top_k > n_experts || N < 0 || N > MAX_N ||
        (int64_t)n_tokens * top_k > MAX_SLOTS || !fits((int64_t)n_tokens * top_k, N))
        return GQ_ERR_SHAPE;
    if (n_experts > 4096) return GQ_ERR_UNSUPPORTED;
    *bytes = gqk_f8_matmul_id_ws_bytes(n_experts, n_tokens, top_k, N, y_dtype, weighted != 0);
    return GQ_OK;
}

gq_status gq_f8_matmul_id(const void* experts, const float* wscales, int32_t n_experts, int64_t N, int64_t K,
                          const int32_t* ids, int32_t n_tokens, int32_t top_k, const void* X, const float* xscales,
                          int64_t ldx, int64_t xs_ld, int32_t x_per_slot, const float* route_w, void* Y,
                          gq_dtype y_dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (y_dtype != GQ_F32 && y_dtype != GQ_BF16) return GQ_ERR_DTYPE;
    if (n_experts < 1 || n_tokens < 0 || top_k < 1 || top_k > n_experts || N < 0 || N > MAX_N || bad_k(K) ||
        (x_per_slot != 0 && x_per_slot != 1) || (int64_t)n_tokens * top_k > MAX_SLOTS)
        return GQ_ERR_SHAPE;
    const int64_t slots = (int64_t)n_tokens * top_k, rows = x_per_slot ? slots : n_tokens;
    if (ldx < K || ldx > MAX_K || xs_ld < rows || !fits(rows, ldx) || !fits(blocks(K), xs_ld) || !fits(slots, N) ||
        !fits(N, K) || !fits(n_experts, N * K))
        return GQ_ERR_SHAPE;
    if (n_experts > 4096) return GQ_ERR_UNSUPPORTED;
    if (n_tokens == 0 || N == 0) return GQ_OK;
    // ids may be NULL: the table already in ws is then used
    if (!Y || !ws || (K > 0 && (!experts || !wscales || !X || !xscales))) return GQ_ERR_NULL;
    if (!aligned16(Y) || !aligned16(ws) || (ids && !aligned16(ids)) || (route_w && !aligned16(route_w)) ||
        (K > 0 && (!aligned16(experts) || !aligned16(wscales) || !aligned16(X) || !aligned16(xscales))))
        return GQ_ERR_ALIGN;
    if (K > 0 && rows > 1 && ldx % 16 != 0) return GQ_ERR_ALIGN;
    if (ws_bytes < gqk_f8_matmul_id_ws_bytes(n_experts, n_tokens, top_k, N, y_dtype, route_w != nullptr))
        return GQ_ERR_WORKSPACE;
    try {
        return from_hip(gqk_f8_matmul_id(static_cast<const uint8_t*>(experts), wscales, n_experts, N, K, ids, n_tokens,
                                         top_k, static_cast<const uint8_t*>(X), xscales, ldx, xs_ld, x_per_slot,
                                         route_w, Y, y_dtype, ws, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_f8_matmul_id_check(const void* ws, hipStream_t stream, int32_t* n_bad_ids) {
    if (!ws || !n_bad_ids) return GQ_ERR_NULL;
    if (!aligned16(ws)) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_f8_matmul_id_bad_count(ws, stream, n_bad_ids));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_route_scored(const void* logits, gq_dtype logits_dtype, int32_t n_tokens, int32_t n_experts,
                          int32_t top_k, gq_score score, const float* bias, int32_t n_groups, int32_t top_groups,
                          gq_group_rank group_rank, int32_t renorm, float scale, int32_t* ids, float* weights,
                          hipStream_t stream) {
    if (logits_dtype != GQ_F32 && logits_dtype != GQ_BF16) return GQ_ERR_DTYPE;
    if (n_tokens < 0 || n_experts < 1 || n_groups < 1 || n_experts % n_groups != 0 || top_groups < 1 ||
        top_groups > n_groups || top_k < 1 || top_k > (int64_t)top_groups * (n_experts / n_groups))
        return GQ_ERR_SHAPE;
    if (n_tokens > MAX_TOKENS) return GQ_ERR_SHAPE;
    if (n_experts > 4096 || top_k > 64 || n_groups > 64) return GQ_ERR_UNSUPPORTED;
    if (score != GQ_SCORE_SOFTMAX && score != GQ_SCORE_SIGMOID) return GQ_ERR_UNSUPPORTED;
    if (group_rank != GQ_GROUP_MAX && group_rank != GQ_GROUP_TOP2) return GQ_ERR_UNSUPPORTED;
    if (n_tokens == 0) return GQ_OK;
    if (!logits || !ids || !weights) return GQ_ERR_NULL;
    if (!aligned16(logits) || !aligned16(ids) || !aligned16(weights) || (bias && !aligned16(bias)))
        return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_route_scored(logits, logits_dtype, n_tokens, n_experts, top_k, score, bias, n_groups,
                                         top_groups, group_rank, renorm != 0, scale, ids, weights, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

}  // extern "C"
