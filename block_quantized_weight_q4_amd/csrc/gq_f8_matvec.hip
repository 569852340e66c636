// gq_f8_matvec.hip -- decode product of 1..16 fp32 / bf16 vectors with
// block-scaled e4m3 weights (gfx950).
//
// y[b][n] = sum over blocks kb of ws[n / 128][kb] * sum_{k in kb} W[n][k] x[b][k].
// Bound by HBM: every weight byte is read once.  One vector is multiplied on the
// vector unit; two and more on the matrix cores (gq_f8_stream.h), with the
// weights widened to bf16 (exact) and fp32 vectors split in three.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_device.h"
#include "gq_f8_internal.h"
#include "gq_f8_stream.h"

using namespace gqf8;

namespace {

template <int NT, int W, int XM, int XR, typename TY>
__global__ __launch_bounds__(64 * W) void k_f8_matvec(const uint8_t* __restrict__ Wt, const float* __restrict__ ws,
                                                      int64_t N, int64_t K, const uint8_t* __restrict__ x, int batch,
                                                      TY* __restrict__ y) {
    using S = Stream<1, NT, XM, XR>;
    constexpr int RING = W * (S::BYTES + S::PARTS), JOIN = W * NT * 1024;
    __shared__ __align__(16) uint8_t smem[RING > JOIN ? RING : JOIN];
    stream_tile<1, NT, W, XM, XR, TY>(
        Wt, ws, (int64_t)blockIdx.x * (16 * NT), N, K, x, nullptr, K * (XM == X_BF16 ? 2 : 4), 0, batch, (N & 3) == 0,
        [&](int i) { return i < batch ? i : batch - 1; }, [&](int i) { return y + (int64_t)i * N; }, smem);
}

// One vector: it would fill one of the matrix cores' columns, or three with an
// fp32 one's parts, and multiplying it in fp32 on the vector unit costs less
// than splitting it (19456 x 2560: 9.4 against 11.5 us; 1024 x 17408: 6.2
// against 15.3 us; two vectors: 5120 x 17408 30.9 against 23.1 us).  A
// workgroup owns R rows; its four wavefronts take 1024 inputs each in turn, lane
// l 16 of them, so that a load instruction reads 1 KB of one row.  No loads
// ahead: the wavefronts hide each other's (two 1024s in flight each: 12.8 us).
// R = 4: two rows read x twice as often (34816 x 5120: 39.7 against 32.4 us),
// eight leave too few wavefronts (5120 x 17408: 22.6 against 16.1 us).
constexpr int R = 4, DOT_WAVES = 4;

template <typename TX, typename TY>
__global__ __launch_bounds__(64 * DOT_WAVES) void k_f8_dot(const uint8_t* __restrict__ Wt,
                                                           const float* __restrict__ ws, int64_t N, int64_t K,
                                                           const TX* __restrict__ x, TY* __restrict__ y) {
    __shared__ float part[DOT_WAVES][R];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * R;
    const int KB = (int)((K + BLK - 1) / BLK);
    const int64_t rows = N - n0 < R ? N - n0 : R;
    const Rsrc wr = make_rsrc(Wt + n0 * K, rows * K);
    const Rsrc xr = make_rsrc(x, K * (int64_t)sizeof(TX));
    const Rsrc sr = make_rsrc(ws + (n0 / BLK) * KB, (int64_t)KB * 4);  // (R rows lie in one block of 128)
    constexpr int XL = sizeof(TX);                                     // 16-byte loads of 16 inputs
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.0f;
    const int J = (int)((K + 1023) / 1024);
    for (int j = wave; j < J; j += DOT_WAVES) {
        // (past the row's end: zeros)
        const int k = j * 1024 + 16 * lane;
        u32x4 w[R], xv[XL];
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = bld16(wr, within((uint32_t)(r * K + k), k, (int)K));
#pragma unroll
        for (int i = 0; i < XL; ++i) xv[i] = bld16(xr, within((uint32_t)(k * XL + 16 * i), k, (int)K));
        const float s = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(sr, (int)within((uint32_t)(k / BLK * 4), k, (int)K), 0, 0));
        float xf[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // (a copy first: a bit_cast of a vector's element takes element 0)
            const uint32_t u = XL == 4 ? xv[i / 4][i % 4] : xv[i / 8][(i % 8) / 2];
            xf[i] = __builtin_bit_cast(float, XL == 4 ? u : i & 1 ? u & 0xffff0000u : u << 16);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float d = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[r][i], false);
                const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[r][i], true);
                d = __builtin_fmaf(lo.x, xf[4 * i], d);
                d = __builtin_fmaf(lo.y, xf[4 * i + 1], d);
                d = __builtin_fmaf(hi.x, xf[4 * i + 2], d);
                d = __builtin_fmaf(hi.y, xf[4 * i + 3], d);
            }
            acc[r] = __builtin_fmaf(s, d, acc[r]);
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
    if (row < rows) store_as(y + n0 + row, (part[0][row] + part[1][row]) + (part[2][row] + part[3][row]));
}

template <typename TX>
hipError_t dot(const uint8_t* W, const float* ws, int64_t N, int64_t K, const void* x, void* y, int y_dtype,
               hipStream_t s) {
    const dim3 grid((unsigned)((N + R - 1) / R)), block(64 * DOT_WAVES);
    if (y_dtype == gqd::DT_F32)
        hipLaunchKernelGGL((k_f8_dot<TX, float>), grid, block, 0, s, W, ws, N, K, static_cast<const TX*>(x),
                           static_cast<float*>(y));
    else
        hipLaunchKernelGGL((k_f8_dot<TX, uint16_t>), grid, block, 0, s, W, ws, N, K, static_cast<const TX*>(x),
                           static_cast<uint16_t*>(y));
    return hipGetLastError();
}

template <int NT, int W, int XM, int XR, typename TY>
hipError_t launch_y(const uint8_t* Wt, const float* ws, int64_t N, int64_t K, const void* x, int batch, TY* y,
                    hipStream_t s) {
    hipLaunchKernelGGL((k_f8_matvec<NT, W, XM, XR, TY>), dim3((unsigned)((N + 16 * NT - 1) / (16 * NT))),
                       dim3(64 * W), 0, s, Wt, ws, N, K, static_cast<const uint8_t*>(x), batch, y);
    return hipGetLastError();
}

template <int NT, int W, int XM, typename TY>
hipError_t launch_x(const uint8_t* Wt, const float* ws, int64_t N, int64_t K, const void* x, int batch, TY* y,
                    hipStream_t s) {
    if (batch <= 4) return launch_y<NT, W, XM, 4, TY>(Wt, ws, N, K, x, batch, y, s);
    if (batch <= 8) return launch_y<NT, W, XM, 8, TY>(Wt, ws, N, K, x, batch, y, s);
    return launch_y<NT, W, XM, 16, TY>(Wt, ws, N, K, x, batch, y, s);
}

template <int NT, int W>
hipError_t launch(const uint8_t* Wt, const float* ws, int64_t N, int64_t K, const void* x, int x_dtype, int batch,
                  void* y, int y_dtype, hipStream_t s) {
    auto* yf = static_cast<float*>(y);
    auto* yb = static_cast<uint16_t*>(y);
    const bool xf32 = x_dtype == gqd::DT_F32, yf32 = y_dtype == gqd::DT_F32;
    if (xf32 && yf32) return launch_x<NT, W, X_F32>(Wt, ws, N, K, x, batch, yf, s);
    if (xf32) return launch_x<NT, W, X_F32>(Wt, ws, N, K, x, batch, yb, s);
    if (yf32) return launch_x<NT, W, X_BF16>(Wt, ws, N, K, x, batch, yf, s);
    return launch_x<NT, W, X_BF16>(Wt, ws, N, K, x, batch, yb, s);
}

}  // namespace

hipError_t gqk_f8_matvec(const uint8_t* W, const float* ws, int64_t N, int64_t K, const void* x, int x_dtype,
                         int batch, void* y, int y_dtype, hipStream_t s) {
    if (batch == 1 && grid_ok((N + R - 1) / R, 64 * DOT_WAVES))
        return x_dtype == gqd::DT_F32 ? dot<float>(W, ws, N, K, x, y, y_dtype, s)
                                      : dot<uint16_t>(W, ws, N, K, x, y, y_dtype, s);
    // NT: 32 rows a workgroup read x half as often as 16 do (5120 x 17408, 16
    // vectors: 22.9 against 30.0 us), but below 128 workgroups 16 rows are
    // faster (2560 x 9728, 8 vectors: 7.0 against 7.6 us).  W: eight wavefronts
    // for long rows (5120 x 17408: 22.9 against 28.0 us), four where each would
    // have few blocks (19456 x 2560: 10.2 against 11.0 us).
    if (N <= 32 * 128) return launch<1, 8>(W, ws, N, K, x, x_dtype, batch, y, y_dtype, s);
    if (K >= 32 * BLK) return launch<2, 8>(W, ws, N, K, x, x_dtype, batch, y, y_dtype, s);
    return launch<2, 4>(W, ws, N, K, x, x_dtype, batch, y, y_dtype, s);
}
