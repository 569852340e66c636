// gq_g4_vectors.h -- decode product of up to 16 vectors with 4-bit weights on the
// matrix cores (gfx950); each type of vectors is compiled in a file of its own.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_g4_device.h"
#include "gq_g4_internal.h"
#include "gq_g4_stream.h"

namespace gqg4 {

template <typename X, bool ZP, int G, int NT, int W, int XR>
__global__ __launch_bounds__(64 * W) void k_g4_vectors(G4Weights wt, const void* __restrict__ x, int batch,
                                                       void* __restrict__ y, int y_dtype) {
    using S = StreamSize<X, NT, XR>;
    __shared__ __align__(16) uint8_t smem[W * (S::BYTES > S::JOIN ? S::BYTES : S::JOIN)];
    stream_tile<X, ZP, G, NT, W, XR>(wt, (int64_t)blockIdx.x * (16 * NT), x, wt.K, batch, smem,
                                     [&](int i, int64_t n, f32x4 v, int c) { store_as(y, i * wt.N + n, y_dtype, v, c); });
}

// (at most MOST wavefronts: as many as 160 KB of LDS hold)
template <typename X, bool ZP, int G, int NT, int MOST, int XR>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    constexpr int EACH = StreamSize<X, NT, XR>::BYTES, W = MOST * EACH <= 163840 ? MOST : MOST / 2;
    static_assert(W * EACH <= 163840, "LDS");
    const int64_t groups = (w.N + 16 * NT - 1) / (16 * NT);
    if (!grid_ok(groups, 64 * W)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_g4_vectors<X, ZP, G, NT, W, XR>), dim3((unsigned)groups), dim3(64 * W), 0, s, w, x, batch, y,
                       y_dtype);
    return hipGetLastError();
}

template <typename X, bool ZP, int G, int NT, int W>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    if (batch <= 4) return vectors<X, ZP, G, NT, W, 4>(w, x, batch, y, y_dtype, s);
    // (eight fp32 vectors, split by one lane for all: 19456 x 2560 24 us, as sixteen 21 us)
    if (X::SIZE == 2 && batch <= 8) return vectors<X, ZP, G, NT, W, X::SIZE == 2 ? 8 : 16>(w, x, batch, y, y_dtype, s);
    return vectors<X, ZP, G, NT, W, 16>(w, x, batch, y, y_dtype, s);
}

// Rows of W a workgroup and wavefronts: 32 rows read X half as often as 16 (34816 x
// 5120, 16 bf16 vectors: 32 and 39 us), but below 4096 rows 16 make more workgroups
// (2560 x 9728, 8 vectors: 7.1 and 10.1 us) and up to 4 vectors have little X to read
// (19456 x 2560, 1 vector: 8.9 and 9.9 us).  5120 rows, which 16 would spread over all
// CUs, take 32 too (5120 x 17408, 8 vectors: 14.8 and 15.8 us, 16 vectors: 16.8 and 20.3;
// from HBM alone 18.2 and 21.9 with 8).  Up to 8192 rows eight wavefronts a
// workgroup (5120 x 17408, 8 vectors: 18.4 us, with four 19.3; 2560 x 9728, 1 vector:
// 6.6, 9.1), above that four, each with more blocks (19456 x 2560, 16 vectors: 13 us,
// with eight 18).
template <typename X, bool ZP, int G>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    if (w.N <= 4096) return vectors<X, ZP, G, 1, 8>(w, x, batch, y, y_dtype, s);
    if (w.N <= 8192) return vectors<X, ZP, G, 2, 8>(w, x, batch, y, y_dtype, s);
    if (X::SIZE == 2 && batch <= 4) return vectors<X, ZP, G, 1, 4, 4>(w, x, batch, y, y_dtype, s);
    return vectors<X, ZP, G, 2, 4>(w, x, batch, y, y_dtype, s);
}

template <typename X, bool ZP>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    if (w.group == 32) return vectors<X, ZP, 32>(w, x, batch, y, y_dtype, s);
    if (w.group == 64) return vectors<X, ZP, 64>(w, x, batch, y, y_dtype, s);
    return vectors<X, ZP, 128>(w, x, batch, y, y_dtype, s);
}

template <typename X>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    return w.zeros ? vectors<X, true>(w, x, batch, y, y_dtype, s) : vectors<X, false>(w, x, batch, y, y_dtype, s);
}

}  // namespace gqg4
