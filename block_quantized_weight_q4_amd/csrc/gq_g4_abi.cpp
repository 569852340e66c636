// gq_g4_abi.cpp -- the extern "C" boundary of gq_g4.h: argument validation
// (before any HIP call) and dispatch to the kernel launchers.
#include "../../include/gq_g4.h"

#include <hip/hip_runtime.h>

#include "gq_g4_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gq_status from_hip(hipError_t e) { return e == hipSuccess ? GQ_OK : GQ_ERR_LAUNCH; }

// Largest element count of any operand, longest row (as in gq_abi.cpp), most
// rows of X (tiles are counted in 32 bits) and of W (a launch has at most 2^32
// threads).
constexpr int64_t MAX_ELEMS = (int64_t)1 << 40;
constexpr int64_t MAX_K = (int64_t)1 << 22;
constexpr int64_t MAX_ROWS = ((int64_t)1 << 31) - 256;
constexpr int64_t MAX_N = ((int64_t)1 << 28) - 256;

// rows x stride elements within MAX_ELEMS (both already known to be >= 0)
bool fits(int64_t rows, int64_t stride) { return rows == 0 || stride <= MAX_ELEMS / rows; }

gq_status check_weights(gq_dtype s_dtype, int32_t group, int64_t N, int64_t K) {
    if (s_dtype != GQ_BF16 && s_dtype != GQ_F16) return GQ_ERR_DTYPE;
    if (N < 0 || N > MAX_N || K < 0 || K % 32 != 0 || K > MAX_K || !fits(N, K)) return GQ_ERR_SHAPE;
    if (group != 32 && group != 64 && group != 128) return GQ_ERR_UNSUPPORTED;
    return GQ_OK;
}

gq_status check_rows(int64_t N, int64_t K, int64_t M, int32_t n_experts, const int32_t* offsets) {
    if (M < 0 || M > MAX_ROWS || n_experts < 1 || (!offsets && n_experts != 1)) return GQ_ERR_SHAPE;
    if (n_experts > 4096) return GQ_ERR_UNSUPPORTED;
    return fits(n_experts, N * K) ? GQ_OK : GQ_ERR_SHAPE;
}

G4Weights weights(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group, int64_t N,
                  int64_t K) {
    return G4Weights{static_cast<const uint8_t*>(W), static_cast<const uint16_t*>(scales),
                     static_cast<const uint8_t*>(zeros), N, K, group, s_dtype == GQ_F16};
}

}  // namespace

extern "C" {

gq_status gq_g4_matvec(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group,
                       int64_t N, int64_t K, const void* x, gq_dtype x_dtype, int32_t batch, void* y,
                       gq_dtype y_dtype, hipStream_t stream) {
    if (x_dtype != GQ_F32 && x_dtype != GQ_BF16 && x_dtype != GQ_F16) return GQ_ERR_DTYPE;
    if (y_dtype != GQ_F32 && y_dtype != GQ_BF16 && y_dtype != GQ_F16) return GQ_ERR_DTYPE;
    const gq_status st = check_weights(s_dtype, group, N, K);
    if (st != GQ_OK) return st;
    if (batch < 1) return GQ_ERR_SHAPE;
    if (batch > 16) return GQ_ERR_UNSUPPORTED;
    if (N == 0) return GQ_OK;
    if (!y || (K > 0 && (!W || !scales || !x))) return GQ_ERR_NULL;
    if (!aligned16(y) || (K > 0 && (!aligned16(W) || !aligned16(scales) || !aligned16(x) || !aligned16(zeros))))
        return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_g4_matvec(weights(W, scales, s_dtype, zeros, group, N, K), x, x_dtype, batch, y, y_dtype,
                                      stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_g4_matmul(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group,
                       int64_t N, int64_t K, const void* X, gq_dtype x_dtype, int64_t M, int64_t ldx, void* Y,
                       gq_dtype y_dtype, int64_t ldy, int32_t n_experts, const int32_t* offsets,
                       hipStream_t stream) {
    if (x_dtype != GQ_BF16 && x_dtype != GQ_F16) return GQ_ERR_DTYPE;
    if (y_dtype != GQ_F32 && y_dtype != x_dtype) return GQ_ERR_DTYPE;
    gq_status st = check_weights(s_dtype, group, N, K);
    if (st == GQ_OK) st = check_rows(N, K, M, n_experts, offsets);
    if (st != GQ_OK) return st;
    // (128 rows of X are addressed in 31 bits)
    if (ldx < K || ldx > MAX_K || ldy < N || !fits(M, ldx) || !fits(M, ldy)) return GQ_ERR_SHAPE;
    if (M == 0 || N == 0) return GQ_OK;
    if (!Y || (K > 0 && (!W || !scales || !X))) return GQ_ERR_NULL;
    if (!aligned16(Y) || !aligned16(offsets) ||
        (K > 0 && (!aligned16(W) || !aligned16(scales) || !aligned16(X) || !aligned16(zeros))))
        return GQ_ERR_ALIGN;
    if (K > 0 && M > 1 && ldx % 8 != 0) return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_g4_matmul(weights(W, scales, s_dtype, zeros, group, N, K), X, x_dtype, M, ldx, Y, y_dtype,
                                      ldy, n_experts, offsets, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

gq_status gq_g4_matmul_dx(const void* W, const void* scales, gq_dtype s_dtype, const void* zeros, int32_t group,
                          int64_t N, int64_t K, const void* dY, gq_dtype dtype, int64_t M, int64_t lddy, void* dX,
                          int64_t lddx, int32_t n_experts, const int32_t* offsets, hipStream_t stream) {
    if (dtype != GQ_BF16 && dtype != GQ_F16) return GQ_ERR_DTYPE;
    gq_status st = check_weights(s_dtype, group, N, K);
    if (st == GQ_OK) st = check_rows(N, K, M, n_experts, offsets);
    if (st != GQ_OK) return st;
    if (lddy < N || lddx < K || !fits(M, lddy) || !fits(M, lddx)) return GQ_ERR_SHAPE;
    if (M == 0 || K == 0) return GQ_OK;
    if (!dX || (N > 0 && (!W || !scales || !dY))) return GQ_ERR_NULL;
    if (!aligned16(dX) || !aligned16(offsets) ||
        (N > 0 && (!aligned16(W) || !aligned16(scales) || !aligned16(dY) || !aligned16(zeros))))
        return GQ_ERR_ALIGN;
    try {
        return from_hip(gqk_g4_matmul_dx(weights(W, scales, s_dtype, zeros, group, N, K), dY, dtype, M, lddy, dX, lddx,
                                         n_experts, offsets, stream));
    } catch (...) {
        return GQ_ERR_LAUNCH;
    }
}

}  // extern "C"
