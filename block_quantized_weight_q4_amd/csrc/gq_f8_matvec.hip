// gq_f8_matvec.hip -- decode product of 1..16 fp32 / bf16 vectors with
// block-scaled e4m3 weights (gfx950).
//
// y[b][n] = sum over blocks kb of ws[n / 128][kb] * sum_{k in kb} W[n][k] x[b][k].
// Bound by HBM: every weight byte is read once (gq_f8_stream.h).  The matrix
// cores take the product for any number of vectors, with the weights widened
// to bf16 (exact) and fp32 vectors split in two, so that the vector unit has
// little more to do than to widen: for one vector this is as fast as
// multiplying on the vector unit was (19456 x 2560: 10.2 against 10.3 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_device.h"
#include "gq_f8_internal.h"
#include "gq_f8_stream.h"

using namespace gqf8;

namespace {

template <int NT, int W, int D, int XM, int XR, typename TY>
__global__ __launch_bounds__(64 * W) void k_f8_matvec(const uint8_t* __restrict__ Wt, const float* __restrict__ ws,
                                                      int64_t N, int64_t K, const uint8_t* __restrict__ x, int batch,
                                                      TY* __restrict__ y) {
    constexpr int RING = W * D * Stream<1, NT, XM, XR>::BYTES, JOIN = W * NT * 1024;
    __shared__ __align__(16) uint8_t smem[RING > JOIN ? RING : JOIN];
    stream_tile<1, NT, W, D, XM, XR, TY>(
        Wt, ws, (int64_t)blockIdx.x * (16 * NT), N, K, x, nullptr, K * (XM == X_BF16 ? 2 : 4), 0, batch, (N & 3) == 0,
        [&](int i) { return i < batch ? i : batch - 1; }, [&](int i) { return y + (int64_t)i * N; }, smem);
}

template <int NT, int W, int D, int XM, int XR, typename TY>
hipError_t launch_y(const uint8_t* Wt, const float* ws, int64_t N, int64_t K, const void* x, int batch, TY* y,
                    hipStream_t s) {
    hipLaunchKernelGGL((k_f8_matvec<NT, W, D, XM, XR, TY>), dim3((unsigned)((N + 16 * NT - 1) / (16 * NT))),
                       dim3(64 * W), 0, s, Wt, ws, N, K, static_cast<const uint8_t*>(x), batch, y);
    return hipGetLastError();
}

template <int NT, int W, int D, int XM, typename TY>
hipError_t launch_x(const uint8_t* Wt, const float* ws, int64_t N, int64_t K, const void* x, int batch, TY* y,
                    hipStream_t s) {
    if (batch <= 4) return launch_y<NT, W, D, XM, 4, TY>(Wt, ws, N, K, x, batch, y, s);
    if (batch <= 8) return launch_y<NT, W, D, XM, 8, TY>(Wt, ws, N, K, x, batch, y, s);
    return launch_y<NT, W, D, XM, 16, TY>(Wt, ws, N, K, x, batch, y, s);
}

template <int NT, int W, int D>
hipError_t launch(const uint8_t* Wt, const float* ws, int64_t N, int64_t K, const void* x, int x_dtype, int batch,
                  void* y, int y_dtype, hipStream_t s) {
    auto* yf = static_cast<float*>(y);
    auto* yb = static_cast<uint16_t*>(y);
    const bool xf32 = x_dtype == gqd::DT_F32, yf32 = y_dtype == gqd::DT_F32;
    if (xf32 && yf32) return launch_x<NT, W, D, X_F32>(Wt, ws, N, K, x, batch, yf, s);
    if (xf32) return launch_x<NT, W, D, X_F32>(Wt, ws, N, K, x, batch, yb, s);
    if (yf32) return launch_x<NT, W, D, X_BF16>(Wt, ws, N, K, x, batch, yf, s);
    return launch_x<NT, W, D, X_BF16>(Wt, ws, N, K, x, batch, yb, s);
}

}  // namespace

hipError_t gqk_f8_matvec(const uint8_t* W, const float* ws, int64_t N, int64_t K, const void* x, int x_dtype,
                         int batch, void* y, int y_dtype, hipStream_t s) {
    // NT: 32 rows a workgroup read x half as often as 16 do (5120 x 17408, 16
    // vectors: 22.9 against 30.0 us), but below 128 workgroups 16 rows are
    // faster (2560 x 9728, 8 vectors: 7.0 against 7.6 us).  W: eight wavefronts
    // for long rows (5120 x 17408: 22.9 against 28.0 us), four where each would
    // have few blocks (19456 x 2560: 10.2 against 11.0 us).  A ring of one block
    // a wavefront is enough with that many of them (two: 12.0, 22.6 us).
    if (N <= 32 * 128) return launch<1, 8, 1>(W, ws, N, K, x, x_dtype, batch, y, y_dtype, s);
    if (K >= 32 * BLK) return launch<2, 8, 1>(W, ws, N, K, x, x_dtype, batch, y, y_dtype, s);
    return launch<2, 4, 1>(W, ws, N, K, x, x_dtype, batch, y, y_dtype, s);
}
