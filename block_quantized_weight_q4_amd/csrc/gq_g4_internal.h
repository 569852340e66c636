// gq_g4_internal.h -- launchers behind gq_g4.h (arguments validated by the ABI
// layer, gq_g4_abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_internal.h"

// Weights of one call: bytes, scales (bf16 or fp16), zero points (NULL: 8).
struct G4Weights {
    const uint8_t* W;
    const uint16_t* scales;
    const uint8_t* zeros;
    int64_t N, K;
    int group, s_f16;
};

hipError_t gqk_g4_matvec(const G4Weights& w, const void* x, int x_dtype, int batch, void* y, int y_dtype,
                         hipStream_t s);
// The same on the matrix cores, by the type of x.
hipError_t gqk_g4_vectors_bf16(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s);
hipError_t gqk_g4_vectors_f16(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s);
hipError_t gqk_g4_vectors_f32(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s);

// offsets NULL: one matrix
hipError_t gqk_g4_matmul(const G4Weights& w, const void* X, int x_dtype, int64_t M, int64_t ldx, void* Y, int y_dtype,
                         int64_t ldy, int n_experts, const int32_t* offsets, hipStream_t s);
hipError_t gqk_g4_matmul_dx(const G4Weights& w, const void* dY, int dtype, int64_t M, int64_t lddy, void* dX,
                            int64_t lddx, int n_experts, const int32_t* offsets, hipStream_t s);
