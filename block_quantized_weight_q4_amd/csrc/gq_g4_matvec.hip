// gq_g4_matvec.hip -- decode product of 1..16 vectors with 4-bit weights and
// group scales (gfx950).
//
// y[b][n] = sum over groups g of s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) x[b][k].
// Bound by HBM: every weight byte is read once.  One fp32 vector is multiplied
// on the vector unit, others on the matrix cores (gq_g4_stream.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_g4_device.h"
#include "gq_g4_internal.h"

using namespace gqg4;

namespace {

// One vector in fp32: it would fill one of the matrix cores' columns, three with its
// bf16 parts.  A workgroup owns R rows; its wavefronts take 1024 inputs each in turn,
// lane l 16 of them (within one group), so that a load instruction reads 512 bytes of
// one row.  19456 x 2560 (25.7 MB) takes 9.3 us, 10.4 from HBM alone, next to a call's own
// 6.2: a wavefront has one or two turns, so the loads' latency and the sums at the end
// are most of it; 5120 x 17408 (46 MB) 12.8, with x in LDS 22.
template <bool ZP, int R, int W>
__global__ __launch_bounds__(64 * W) void k_g4_dot(G4Weights wt, const float* __restrict__ x, void* __restrict__ y,
                                                   int y_dtype) {
    __shared__ float part[W][R];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t N = wt.N, K = wt.K, row_bytes = K / 2, n0 = (int64_t)blockIdx.x * R;
    const int rows = N - n0 < R ? (int)(N - n0) : R;
    const int KG = (int)((K + wt.group - 1) / wt.group), gshift = __builtin_ctz(wt.group);
    const Rsrc wr = make_rsrc(wt.W + n0 * row_bytes, rows * row_bytes);
    const Rsrc xr = make_rsrc(x, K * 4);
    const Rsrc sr = make_rsrc(wt.scales + n0 * KG, (int64_t)rows * KG * 2);
    const Rsrc zr = make_rsrc(ZP ? wt.zeros + n0 * KG : nullptr, ZP ? (int64_t)rows * KG : 0);
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.0f;
    for (int k = 1024 * wave + 16 * lane; k - 16 * lane < K; k += 1024 * W) {
        // (past the row's end: zeros, the scale's among them)
        const int left = (int)K - k;
        u32x2 w[R];
        uint32_t s[R], z[R];
        u32x4 xv[4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(
                                                 wr, (int)within((uint32_t)(r * row_bytes + k / 2), 0, left), 0, 0));
            const int g = r * KG + (k >> gshift);
            s[r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(sr, (int)within(2u * (uint32_t)g, 0, left), 0, 0);
            if constexpr (ZP)
                z[r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(zr, (int)within((uint32_t)g, 0, left), 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = bld16(xr, within(4u * (uint32_t)k + 16 * i, 0, left));
        float xf[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t u = xv[i / 4][i % 4];  // (a copy first: a bit_cast of a vector's element takes element 0)
            xf[i] = __builtin_bit_cast(float, u);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t z4 = ZP ? zero4(z[r]) : 0u;
            const Centred<ZP> a(w[r].x, z4), b(w[r].y, z4);
            float d = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) d = __builtin_fmaf(a.at(i), xf[i], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) d = __builtin_fmaf(b.at(i), xf[8 + i], d);
            acc[r] = __builtin_fmaf(scale_f32(s[r], wt.s_f16) * Centred<ZP>::UNIT, d, acc[r]);
        }
    }
    // sums over the lanes; each of the first steps halves the rows that a lane holds
    int off = 32;
#pragma unroll
    for (int n = R / 2; n >= 1; n >>= 1, off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float keep = up ? acc[i + n] : acc[i], give = up ? acc[i] : acc[i + n];
            acc[i] = keep + __shfl_xor(give, off, 64);
        }
    }
    for (; off >= 1; off >>= 1) acc[0] += __shfl_xor(acc[0], off, 64);
    // lane bits 5, 4, .. select the row, highest bit first
    if ((lane & (64 / R - 1)) == 0) part[wave][lane / (64 / R)] = acc[0];
    __syncthreads();
    const int row = threadIdx.x;
    if (row < rows) {
        float v = part[0][row];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][row];
        store_as(y, n0 + row, y_dtype, v);
    }
}

template <bool ZP, int R, int W>
hipError_t dot(G4Weights w, const void* x, void* y, int y_dtype, hipStream_t s) {
    // (a launch has fewer than 2^32 threads)
    constexpr int64_t MOST = (int64_t)R << 24;
    const int64_t N = w.N, KG = (w.K + w.group - 1) / w.group;
    for (int64_t n = 0; n < N; n += MOST) {
        w.N = N - n < MOST ? N - n : MOST;
        hipLaunchKernelGGL((k_g4_dot<ZP, R, W>), dim3((unsigned)((w.N + R - 1) / R)), dim3(64 * W), 0, s, w,
                           static_cast<const float*>(x), y, y_dtype);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        w.W += MOST * (w.K / 2);
        w.scales += MOST * KG;
        if (ZP) w.zeros += MOST * KG;
        y = static_cast<uint8_t*>(y) + MOST * (y_dtype == gqd::DT_F32 ? 4 : 2);
    }
    return hipSuccess;
}

template <bool ZP>
hipError_t dot(const G4Weights& w, const void* x, void* y, int y_dtype, hipStream_t s) {
    return dot<ZP, 4, 2>(w, x, y, y_dtype, s);
}

}  // namespace

hipError_t gqk_g4_matvec(const G4Weights& w, const void* x, int x_dtype, int batch, void* y, int y_dtype,
                         hipStream_t s) {
    if (x_dtype == gqd::DT_BF16) return gqk_g4_vectors_bf16(w, x, batch, y, y_dtype, s);
    if (x_dtype == gqd::DT_F16) return gqk_g4_vectors_f16(w, x, batch, y, y_dtype, s);
    if (batch > 1) return gqk_g4_vectors_f32(w, x, batch, y, y_dtype, s);
    return w.zeros ? dot<true>(w, x, y, y_dtype, s) : dot<false>(w, x, y, y_dtype, s);
}
