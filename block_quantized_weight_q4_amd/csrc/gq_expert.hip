// gq_expert.hip -- tokens sorted by expert and back (gfx950): a counting sort by
// one workgroup; one workgroup a token for the rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_device.h"
#include "gq_expert_internal.h"

namespace {

constexpr int MAX_E = 4096;

__global__ __launch_bounds__(1024) void k_sort(const int32_t* __restrict__ ids, int S, int E,
                                               int32_t* __restrict__ offsets, int32_t* __restrict__ place) {
    __shared__ int count[MAX_E];
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < E; e += 1024) count[e] = 0;
    __syncthreads();
    for (int s = tid; s < S; s += 1024) {
        const int id = ids[s];
        if (id >= 0 && id < E) atomicAdd(&count[id], 1);
    }
    __syncthreads();
    if (tid == 0) {
        int sum = 0;
        for (int e = 0; e < E; ++e) {
            const int c = count[e];
            offsets[e] = count[e] = sum;
            sum += c;
        }
        offsets[E] = sum;
    }
    __syncthreads();
    // the first wavefront places 64 slots at a time, in their order
    if (tid >= 64) return;
    for (int s0 = 0; s0 < S; s0 += 64) {
        const int s = s0 + lane, id = s < S ? ids[s] : -1;
        const bool ok = id >= 0 && id < E;
        uint64_t same = __ballot(ok);
        for (int b = 0; b < 12; ++b) {  // (E <= 4096)
            const uint64_t m = __ballot((id >> b) & 1);
            same &= (id >> b) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int base = ok ? count[id] : 0;
        __builtin_amdgcn_wave_barrier();
        if (ok && rank == 0) count[id] = base + __popcll(same);
        if (s < S) place[s] = ok ? base + rank : -1;
    }
}

__device__ __forceinline__ float to_f32(const void* p, int64_t i, int dtype) {
    if (dtype == gqd::DT_F32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return dtype == gqd::DT_BF16 ? gqd::bf2f(u) : gqd::h2f(u);
}

__device__ __forceinline__ void store_f32(void* p, int64_t i, int dtype, float v) {
    if (dtype == gqd::DT_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = dtype == gqd::DT_BF16 ? gqd::f2bf(v) : gqd::f2h(v);
}

template <typename T>
__global__ __launch_bounds__(256) void k_gather(const T* __restrict__ x, int64_t top_k, int64_t D, int64_t ldx,
                                                const int32_t* __restrict__ place, T* __restrict__ xs, int64_t ldxs) {
    const int64_t t = blockIdx.x, S = gridDim.x * top_k;
    for (int64_t d = threadIdx.x; d < D; d += 256) {
        const T v = x[t * ldx + d];
        for (int64_t j = 0; j < top_k; ++j) {
            const int64_t p = place[t * top_k + j];
            if (p >= 0 && p < S) xs[p * ldxs + d] = v;
        }
    }
}

__global__ __launch_bounds__(256) void k_combine(const void* __restrict__ ys, int dtype, int64_t top_k, int64_t D,
                                                 int64_t ldys, const int32_t* __restrict__ place,
                                                 const float* __restrict__ w, void* __restrict__ y, int y_dtype,
                                                 int64_t ldy) {
    const int64_t t = blockIdx.x, S = gridDim.x * top_k;
    for (int64_t d = threadIdx.x; d < D; d += 256) {
        float sum = 0.0f;
        for (int64_t j = 0; j < top_k; ++j) {
            const int64_t p = place[t * top_k + j];
            if (p >= 0 && p < S)
                sum = __builtin_fmaf(w ? w[t * top_k + j] : 1.0f, to_f32(ys, p * ldys + d, dtype), sum);
        }
        store_f32(y, t * ldy + d, y_dtype, sum);
    }
}

// One workgroup a slot.  (dys may be ys: no __restrict__)
__global__ __launch_bounds__(256) void k_combine_grad(const void* dy, int dtype, int64_t top_k, int64_t D,
                                                      int64_t lddy, const void* ys, int64_t ldys,
                                                      const int32_t* __restrict__ place, const float* __restrict__ w,
                                                      void* dys, int64_t lddys, float* __restrict__ dw) {
    __shared__ float part[4];
    const int64_t slot = blockIdx.x, t = slot / top_k, S = gridDim.x, p = place[slot];
    const bool ok = p >= 0 && p < S;
    float sum = 0.0f;
    if (ok) {
        const float f = w ? w[slot] : 1.0f;
        for (int64_t d = threadIdx.x; d < D; d += 256) {
            const float g = to_f32(dy, t * lddy + d, dtype);
            if (dw) sum = __builtin_fmaf(g, to_f32(ys, p * ldys + d, dtype), sum);
            if (dys) store_f32(dys, p * lddys + d, dtype, f * g);
        }
    }
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (dw && threadIdx.x == 0) dw[slot] = (part[0] + part[1]) + (part[2] + part[3]);
}

}  // namespace

hipError_t gqk_expert_sort(const int32_t* ids, int n_tokens, int top_k, int n_experts, int32_t* offsets,
                           int32_t* place, hipStream_t s) {
    hipLaunchKernelGGL(k_sort, dim3(1), dim3(1024), 0, s, ids, n_tokens * top_k, n_experts, offsets, place);
    return hipGetLastError();
}

hipError_t gqk_expert_gather(const void* x, int dtype, int n_tokens, int top_k, int64_t D, int64_t ldx,
                             const int32_t* place, void* xs, int64_t ldxs, hipStream_t s) {
    if (dtype == gqd::DT_F32)
        hipLaunchKernelGGL(k_gather<uint32_t>, dim3(n_tokens), dim3(256), 0, s, static_cast<const uint32_t*>(x), top_k,
                           D, ldx, place, static_cast<uint32_t*>(xs), ldxs);
    else
        hipLaunchKernelGGL(k_gather<uint16_t>, dim3(n_tokens), dim3(256), 0, s, static_cast<const uint16_t*>(x), top_k,
                           D, ldx, place, static_cast<uint16_t*>(xs), ldxs);
    return hipGetLastError();
}

hipError_t gqk_expert_combine(const void* ys, int dtype, int n_tokens, int top_k, int64_t D, int64_t ldys,
                              const int32_t* place, const float* w, void* y, int y_dtype, int64_t ldy,
                              hipStream_t s) {
    hipLaunchKernelGGL(k_combine, dim3(n_tokens), dim3(256), 0, s, ys, dtype, top_k, D, ldys, place, w, y, y_dtype,
                       ldy);
    return hipGetLastError();
}

hipError_t gqk_expert_combine_grad(const void* dy, int dtype, int n_tokens, int top_k, int64_t D, int64_t lddy,
                                   const void* ys, int64_t ldys, const int32_t* place, const float* w, void* dys,
                                   int64_t lddys, float* dw, hipStream_t s) {
    hipLaunchKernelGGL(k_combine_grad, dim3(n_tokens * top_k), dim3(256), 0, s, dy, dtype, top_k, D, lddy, ys, ldys,
                       place, w, dys, lddys, dw);
    return hipGetLastError();
}
