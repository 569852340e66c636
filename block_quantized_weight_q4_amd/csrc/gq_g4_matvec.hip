// gq_g4_matvec.hip -- decode product of 1..16 vectors with 4-bit weights and
// group scales (gfx950).
//
// y[b][n] = sum over groups g of s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) x[b][k].
// Bound by HBM: every weight byte is read once.  One vector is multiplied in fp32
// on the vector unit; two and more on the matrix cores (gq_g4_stream.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_g4_device.h"
#include "gq_g4_internal.h"
#include "gq_g4_stream.h"

using namespace gqg4;

namespace {

// One vector.  16 lanes share a row, each a 16-byte chunk of 32 inputs (within
// one group), so that a load instruction reads 256 bytes of each of four rows;
// a lane has R rows.  x is staged in LDS as fp32, 32-input chunks 144 bytes
// apart (16 lanes read 16 chunks without bank conflicts).  KS of the workgroup's
// four wavefronts split a row's inputs, 512 at a time in turn.
constexpr int DOT_WAVES = 4, XTILE = 8192, XCHUNK = 36;

__device__ __forceinline__ float x_at(const void* x, int64_t i, int dtype) {
    if (dtype == gqd::DT_F32) return static_cast<const float*>(x)[i];
    const uint16_t u = static_cast<const uint16_t*>(x)[i];
    return dtype == gqd::DT_BF16 ? gqd::bf2f(u) : gqd::h2f(u);
}

template <bool ZP, int R, int KS>
__global__ __launch_bounds__(64 * DOT_WAVES) void k_g4_dot(G4Weights wt, const void* __restrict__ x, int x_dtype,
                                                           void* __restrict__ y, int y_dtype) {
    constexpr int ROWS = 4 * R * (DOT_WAVES / KS);  // of a workgroup
    extern __shared__ __align__(16) float xs[];
    __shared__ float part[DOT_WAVES][4 * R];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = wave % KS, sub = lane & 15;
    const int64_t K = wt.K, row_bytes = K / 2;
    const int64_t n0 = (int64_t)blockIdx.x * ROWS;
    const int64_t rows = wt.N - n0 < ROWS ? wt.N - n0 : ROWS;
    const int KG = (int)((K + wt.group - 1) / wt.group), gshift = __builtin_ctz(wt.group / 32);
    const Rsrc wr = make_rsrc(wt.W + n0 * row_bytes, rows * row_bytes);
    const Rsrc sr = make_rsrc(wt.scales + n0 * KG, rows * KG * 2);
    const Rsrc zr = make_rsrc(ZP ? wt.zeros + n0 * KG : nullptr, ZP ? rows * KG : 0);
    const int C = (int)(K / 32);
    const int row0 = (wave / KS) * 4 * R + (lane >> 4);  // this lane's rows: row0 + 4 r
    struct Step {
        u32x4 w[R];
        uint32_t s[R], z[R];
    };
    auto load = [&](int c, Step& t) {
        const uint32_t g = (uint32_t)(c >> gshift);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = (uint32_t)(row0 + 4 * r);
            t.w[r] = bld16(wr, within(row * (uint32_t)row_bytes + 16u * (uint32_t)c, c, C));
            t.s[r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(sr, (int)within((row * KG + g) * 2, c, C), 0, 0);
            if constexpr (ZP)
                t.z[r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(zr, (int)within(row * KG + g, c, C), 0, 0);
        }
    };
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = 0.0f;
    for (int64_t k0 = 0; k0 < K; k0 += XTILE) {
        const int end = (int)((K - k0 < XTILE ? K : k0 + XTILE) / 32);  // chunks of this tile
        int c = (int)(k0 / 32) + 16 * ks + sub;
        Step t;
        load(c, t);
        if (k0) __syncthreads();
        const int n = (int)(K - k0 < XTILE ? K - k0 : XTILE);
        for (int i = 4 * tid; i < n; i += 4 * 64 * DOT_WAVES) {
            f32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = x_at(x, k0 + i + j, x_dtype);
            *reinterpret_cast<f32x4*>(xs + (i >> 5) * XCHUNK + (i & 31)) = v;
        }
        gqd::lds_barrier();
        for (; c - sub < end; c += 16 * KS) {
            Step next;
            load(c + 16 * KS, next);
            if (c < end) {
                const float* xc = xs + (c - (int)(k0 / 32)) * XCHUNK;
                float d[R];
#pragma unroll
                for (int r = 0; r < R; ++r) d[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 lo = *reinterpret_cast<const f32x4*>(xc + 8 * i);
                    const f32x4 hi = *reinterpret_cast<const f32x4*>(xc + 8 * i + 4);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const Centred<ZP> q(t.w[r][i], ZP ? zero4(t.z[r]) : 0u);
#pragma unroll
                        for (int j = 0; j < 4; ++j) d[r] = __builtin_fmaf(q.at(j), lo[j], d[r]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) d[r] = __builtin_fmaf(q.at(4 + j), hi[j], d[r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r] = __builtin_fmaf(scale_f32(t.s[r], wt.s_f16) * Centred<ZP>::UNIT, d[r], acc[r]);
            }
            t = next;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) acc[r] += __shfl_xor(acc[r], off, 64);
    if constexpr (KS == 1) {
        if (sub == 0)
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (row0 + 4 * r < rows) store_as(y, n0 + row0 + 4 * r, y_dtype, acc[r]);
    } else {
        if (sub == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) part[wave][(lane >> 4) + 4 * r] = acc[r];
        __syncthreads();
        if (tid < ROWS && tid < rows) {
            const int w0 = tid / (4 * R) * KS, i = tid % (4 * R);
            float v = part[w0][i];
#pragma unroll
            for (int w = 1; w < KS; ++w) v += part[w0 + w][i];
            store_as(y, n0 + tid, y_dtype, v);
        }
    }
}

template <bool ZP, int R, int KS>
hipError_t dot(const G4Weights& w, const void* x, int x_dtype, void* y, int y_dtype, hipStream_t s) {
    constexpr int ROWS = 4 * R * (DOT_WAVES / KS);
    const int64_t tile = w.K < XTILE ? w.K : XTILE;
    hipLaunchKernelGGL((k_g4_dot<ZP, R, KS>), dim3((unsigned)((w.N + ROWS - 1) / ROWS)), dim3(64 * DOT_WAVES),
                       (size_t)(tile / 32) * XCHUNK * 4, s, w, x, x_dtype, y, y_dtype);
    return hipGetLastError();
}

template <bool ZP>
hipError_t dot(const G4Weights& w, const void* x, int x_dtype, void* y, int y_dtype, hipStream_t s) {
    if (w.N >= 8192) return dot<ZP, 2, 1>(w, x, x_dtype, y, y_dtype, s);
    return dot<ZP, 2, 4>(w, x, x_dtype, y, y_dtype, s);
}

template <typename X, bool ZP, int G, int NT, int W, int XR>
__global__ __launch_bounds__(64 * W) void k_g4_vectors(G4Weights wt, const void* __restrict__ x, int batch,
                                                       void* __restrict__ y, int y_dtype) {
    using S = StreamSize<X, NT, XR>;
    __shared__ __align__(16) uint8_t smem[W * (S::BYTES > S::JOIN ? S::BYTES : S::JOIN)];
    stream_tile<X, ZP, G, NT, W, XR>(wt, (int64_t)blockIdx.x * (16 * NT), x, wt.K, batch, smem,
                                     [&](int i, int64_t n, float v) { store_as(y, i * wt.N + n, y_dtype, v); });
}

template <typename X, bool ZP, int G, int NT, int W, int XR>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    hipLaunchKernelGGL((k_g4_vectors<X, ZP, G, NT, W, XR>), dim3((unsigned)((w.N + 16 * NT - 1) / (16 * NT))),
                       dim3(64 * W), 0, s, w, x, batch, y, y_dtype);
    return hipGetLastError();
}

template <typename X, bool ZP, int G, int NT, int W>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    if (batch <= 4) return vectors<X, ZP, G, NT, W, 4>(w, x, batch, y, y_dtype, s);
    if (batch <= 8) return vectors<X, ZP, G, NT, W, 8>(w, x, batch, y, y_dtype, s);
    return vectors<X, ZP, G, NT, W, 16>(w, x, batch, y, y_dtype, s);
}

template <typename X, bool ZP, int G>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    if (w.N <= 32 * 128) return vectors<X, ZP, G, 1, 4>(w, x, batch, y, y_dtype, s);
    return vectors<X, ZP, G, 2, 4>(w, x, batch, y, y_dtype, s);
}

template <typename X, bool ZP>
hipError_t vectors(const G4Weights& w, const void* x, int batch, void* y, int y_dtype, hipStream_t s) {
    if (w.group == 32) return vectors<X, ZP, 32>(w, x, batch, y, y_dtype, s);
    if (w.group == 64) return vectors<X, ZP, 64>(w, x, batch, y, y_dtype, s);
    return vectors<X, ZP, 128>(w, x, batch, y, y_dtype, s);
}

template <bool ZP>
hipError_t matvec(const G4Weights& w, const void* x, int x_dtype, int batch, void* y, int y_dtype, hipStream_t s) {
    if (batch == 1) return dot<ZP>(w, x, x_dtype, y, y_dtype, s);
    if (x_dtype == gqd::DT_F32) return vectors<XF32, ZP>(w, x, batch, y, y_dtype, s);
    if (x_dtype == gqd::DT_BF16) return vectors<XBf16, ZP>(w, x, batch, y, y_dtype, s);
    return vectors<XF16, ZP>(w, x, batch, y, y_dtype, s);
}

}  // namespace

hipError_t gqk_g4_matvec(const G4Weights& w, const void* x, int x_dtype, int batch, void* y, int y_dtype,
                         hipStream_t s) {
    return w.zeros ? matvec<true>(w, x, x_dtype, batch, y, y_dtype, s)
                   : matvec<false>(w, x, x_dtype, batch, y, y_dtype, s);
}
