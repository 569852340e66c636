// gq_f8_internal.h -- launchers behind gq_f8.h (arguments validated by the
// ABI layer, gq_f8_abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gq_internal.h"

hipError_t gqk_f8_quant(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx, int pow2, uint8_t* q,
                        int64_t ldq, float* scales, int64_t s_ld, hipStream_t s);
hipError_t gqk_f8_glu_quant(const void* g, const void* u, int dtype, int64_t M, int64_t K, int64_t ldg, int64_t ldu,
                            int act, int pow2, uint8_t* q, int64_t ldq, float* scales, int64_t s_ld, hipStream_t s);

hipError_t gqk_f8_matvec(const uint8_t* W, const float* ws, int64_t N, int64_t K, const void* x, int x_dtype,
                         int batch, void* y, int y_dtype, hipStream_t s);

hipError_t gqk_f8_matmul(const uint8_t* W, const float* ws, int64_t N, int64_t K, const uint8_t* X, const float* xs,
                         int64_t M, int64_t ldx, int64_t xs_ld, void* Y, int y_dtype, int64_t ldy, hipStream_t s);

// Workspace layout is private to gq_f8_matmul.hip.
size_t gqk_f8_matmul_id_ws_bytes(int n_experts, int n_tokens, int top_k, int64_t N, int y_dtype, int weighted);
hipError_t gqk_f8_matmul_id(const uint8_t* W, const float* wsc, int n_experts, int64_t N, int64_t K,
                            const int32_t* ids, int n_tokens, int top_k, const uint8_t* X, const float* xs,
                            int64_t ldx, int64_t xs_ld, int x_per_slot, const float* route_w, void* Y, int y_dtype,
                            void* ws, hipStream_t s);
hipError_t gqk_f8_matmul_id_bad_count(const void* ws, hipStream_t s, int32_t* n_bad);

hipError_t gqk_route_scored(const void* logits, int dtype, int n_tokens, int n_experts, int top_k, int score,
                            const float* bias, int n_groups, int top_groups, int group_rank, int renorm, float scale,
                            int32_t* ids, float* weights, hipStream_t s);
