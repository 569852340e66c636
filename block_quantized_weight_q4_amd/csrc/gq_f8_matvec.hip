// gq_f8_matvec.hip -- decode product of 1..16 fp32 / bf16 vectors with
// block-scaled e4m3 weights (gfx950).
//
// y[b][n] = sum over blocks kb of ws[n / 128][kb] * sum_{k in kb} W[n][k] x[b][k].
// One wavefront per row: 16-byte weight loads, fp32 multiply-adds.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_device.h"
#include "gq_f8_internal.h"

using namespace gqf8;

namespace {

template <typename TX, typename TY>
__global__ __launch_bounds__(256) void k_f8_matvec(const uint8_t* __restrict__ W, const float* __restrict__ ws,
                                                   int64_t N, int64_t K, const TX* __restrict__ x, int batch,
                                                   TY* __restrict__ y) {
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= N) return;
    const int64_t KB = (K + BLK - 1) / BLK;
    float acc[16];
#pragma unroll
    for (int b = 0; b < 16; ++b) acc[b] = 0.0f;
    for (int64_t k = 16 * lane; k < K; k += 1024) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(W + n * K + k);
        const float s = ws[(n / BLK) * KB + k / BLK];
        float f[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            f[4 * i] = lo.x;
            f[4 * i + 1] = lo.y;
            f[4 * i + 2] = hi.x;
            f[4 * i + 3] = hi.y;
        }
#pragma unroll
        for (int b = 0; b < 16; ++b) {
            if (b >= batch) continue;
            float t = 0.0f;
            for (int i = 0; i < 16; ++i) {
                float xv;
                if constexpr (sizeof(TX) == 4) xv = x[b * K + k + i];
                else xv = gqd::bf2f(x[b * K + k + i]);
                t = __builtin_fmaf(f[i], xv, t);
            }
            acc[b] = __builtin_fmaf(s, t, acc[b]);
        }
    }
#pragma unroll
    for (int b = 0; b < 16; ++b) {
        if (b >= batch) continue;
        float v = acc[b];
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
        if (lane == 0) store_as(y + b * N + n, v);
    }
}

}  // namespace

hipError_t gqk_f8_matvec(const uint8_t* W, const float* ws, int64_t N, int64_t K, const void* x, int x_dtype,
                         int batch, void* y, int y_dtype, hipStream_t s) {
    const dim3 grid((unsigned)((N + 3) / 4));
    const auto* xf = static_cast<const float*>(x);
    const auto* xb = static_cast<const uint16_t*>(x);
    auto* yf = static_cast<float*>(y);
    auto* yb = static_cast<uint16_t*>(y);
    if (x_dtype == gqd::DT_F32 && y_dtype == gqd::DT_F32)
        hipLaunchKernelGGL((k_f8_matvec<float, float>), grid, dim3(256), 0, s, W, ws, N, K, xf, batch, yf);
    else if (x_dtype == gqd::DT_F32)
        hipLaunchKernelGGL((k_f8_matvec<float, uint16_t>), grid, dim3(256), 0, s, W, ws, N, K, xf, batch, yb);
    else if (y_dtype == gqd::DT_F32)
        hipLaunchKernelGGL((k_f8_matvec<uint16_t, float>), grid, dim3(256), 0, s, W, ws, N, K, xb, batch, yf);
    else
        hipLaunchKernelGGL((k_f8_matvec<uint16_t, uint16_t>), grid, dim3(256), 0, s, W, ws, N, K, xb, batch, yb);
    return hipGetLastError();
}
