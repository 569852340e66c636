// gq_g4_dx.hip -- gradient of the products with 4-bit weights with respect to X
// (gfx950): one thread an output.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_device.h"
#include "gq_g4_internal.h"

namespace {

__device__ __forceinline__ float to_f32(const void* p, int64_t i, int dtype) {
    if (dtype == gqd::DT_F32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return dtype == gqd::DT_BF16 ? gqd::bf2f(u) : gqd::h2f(u);
}

__device__ __forceinline__ void store_f32(void* p, int64_t i, int dtype, float v) {
    if (dtype == gqd::DT_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = dtype == gqd::DT_BF16 ? gqd::f2bf(v) : gqd::f2h(v);
}

__device__ __forceinline__ float scale_of(const G4Weights& w, int64_t i) {
    return w.s_f16 ? gqd::h2f(w.scales[i]) : gqd::bf2f(w.scales[i]);
}

// Expert of row m, -1 if it has none; every index stays in range whatever offsets hold.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int n_experts, int64_t m) {
    if (!offsets) return 0;
    int lo = 0, hi = n_experts;  // the first e with offsets[e + 1] > m
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (offsets[mid + 1] > m) hi = mid;
        else lo = mid + 1;
    }
    return lo < n_experts && offsets[lo] <= m ? lo : -1;
}

__global__ __launch_bounds__(256) void k_g4_dx(G4Weights w, const void* __restrict__ dY, int dtype, int64_t M,
                                               int64_t lddy, void* __restrict__ dX, int64_t lddx, int n_experts,
                                               const int32_t* __restrict__ offsets) {
    const int64_t groups = (w.K + w.group - 1) / w.group;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < M * w.K; i += gridDim.x * 256ll) {
        const int64_t m = i / w.K, k = i % w.K, b = k / w.group;
        const int e = expert_of(offsets, n_experts, m);
        if (e < 0) continue;
        float acc = 0.0f;
        for (int64_t n = 0; n < w.N; ++n) {
            const int64_t row = e * w.N + n;
            const int z = w.zeros ? w.zeros[row * groups + b] & 15 : 8;
            const int q = (w.W[row * (w.K / 2) + k / 2] >> (4 * (k & 1))) & 15;
            acc = __builtin_fmaf(scale_of(w, row * groups + b) * (float)(q - z), to_f32(dY, m * lddy + n, dtype), acc);
        }
        store_f32(dX, m * lddx + k, dtype, acc);
    }
}

dim3 grid_for(int64_t n) { return dim3((unsigned)((n + 255) / 256 < 65536 ? (n + 255) / 256 : 65536)); }

}  // namespace

hipError_t gqk_g4_matmul_dx(const G4Weights& w, const void* dY, int dtype, int64_t M, int64_t lddy, void* dX,
                            int64_t lddx, int n_experts, const int32_t* offsets, hipStream_t s) {
    hipLaunchKernelGGL(k_g4_dx, grid_for(M * w.K), dim3(256), 0, s, w, dY, dtype, M, lddy, dX, lddx, n_experts,
                       offsets);
    return hipGetLastError();
}
