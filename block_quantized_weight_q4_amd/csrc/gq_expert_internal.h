// gq_expert_internal.h -- launchers behind gq_expert.h (arguments validated by
// the ABI layer, gq_expert_abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_internal.h"

hipError_t gqk_expert_sort(const int32_t* ids, int n_tokens, int top_k, int n_experts, int32_t* offsets,
                           int32_t* place, hipStream_t s);
hipError_t gqk_expert_gather(const void* x, int dtype, int n_tokens, int top_k, int64_t D, int64_t ldx,
                             const int32_t* place, void* xs, int64_t ldxs, hipStream_t s);
hipError_t gqk_expert_combine(const void* ys, int dtype, int n_tokens, int top_k, int64_t D, int64_t ldys,
                              const int32_t* place, const float* w, void* y, int y_dtype, int64_t ldy,
                              hipStream_t s);
hipError_t gqk_expert_combine_grad(const void* dy, int dtype, int n_tokens, int top_k, int64_t D, int64_t lddy,
                                   const void* ys, int64_t ldys, const int32_t* place, const float* w, void* dys,
                                   int64_t lddys, float* dw, hipStream_t s);
