// gq_f8_quant.hip -- activations to e4m3 with one fp32 scale per 128 inputs of
// a row: gq_f8_quant, and gq_f8_glu_quant for h = act(g) * u (gfx950).
//
// Mathematics: s = max|x| / 448 (at least 2^-64, or the power of two above),
// q = e4m3(fp32(x / s)).  The quotient is formed from the correctly rounded
// reciprocal r of s by one correction, y = x r, y + (x - y s) r, which gives
// the correctly rounded x / s (Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990); 2^-64 <= s <= 2^120 keeps
// every term normal wherever the result is not 0.
//
// Bound by HBM: each input is read once and each byte written once.  Eight
// lanes share a group: each holds 16 inputs (two or four 16-byte loads, one
// 16-byte store) and three DPP / xor steps give the group's maximum.  The
// maximum is taken over the magnitudes' bit patterns, where infinities and
// NaNs sort above every number and so cannot be lost.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_device.h"
#include "gq_f8_internal.h"

using namespace gqf8;

namespace {

constexpr float MIN_SCALE = 0x1p-64f;
constexpr int THREADS = 256, GPB = THREADS / 8;  // groups per workgroup

struct f32_t {
    static constexpr int SIZE = 4;
};
struct bf16_t {
    static constexpr int SIZE = 2;
};
struct f16_t {
    static constexpr int SIZE = 2;
};

// 16 consecutive inputs as fp32.
template <typename T>
__device__ __forceinline__ void load16(const uint8_t* p, float (&v)[16]) {
    if constexpr (T::SIZE == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(p + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = a[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 a = *reinterpret_cast<const u32x4*>(p + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (__is_same(T, bf16_t)) {
                    v[8 * i + 2 * j] = __builtin_bit_cast(float, a[j] << 16);
                    v[8 * i + 2 * j + 1] = __builtin_bit_cast(float, a[j] & 0xffff0000u);
                } else {
                    v[8 * i + 2 * j] = gqd::h2f(a[j] & 0xffffu);
                    v[8 * i + 2 * j + 1] = gqd::h2f(a[j] >> 16);
                }
            }
        }
    }
}

// Scale and e4m3 bytes of this lane's 16 inputs of a group (8 lanes).
__device__ __forceinline__ u32x4 quantise(const float (&v)[16], int pow2, float& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
        top = b > top ? b : top;
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, off, 64);
        top = o > top ? o : top;
    }
    const bool finite = top < 0x7f800000u;
    float s = finite ? __builtin_bit_cast(float, top) / 448.0f : 1.0f;
    if (pow2) {
        const uint32_t b = __builtin_bit_cast(uint32_t, s);  // (subnormal s ends at MIN_SCALE)
        s = __builtin_bit_cast(float, (b + 0x7fffffu) & 0x7f800000u);
    }
    s = s > MIN_SCALE ? s : MIN_SCALE;
    const float r = 1.0f / s;
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = finite ? v[4 * j + i] : 0.0f;
            const float y0 = x * r;
            y[i] = __builtin_fmaf(__builtin_fmaf(-y0, s, x), r, y0);
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
        q[j] = (uint32_t)w;
    }
    scale = finite ? s : __builtin_nanf("");
    return q;
}

// Group i of the flat order (group-of-row b, row m) with m fastest: the scales
// of neighbouring groups are neighbours in memory.
template <typename T, bool GLU>
__global__ __launch_bounds__(THREADS) void k_f8_quant(const uint8_t* __restrict__ x, const uint8_t* __restrict__ u,
                                                      int64_t M, int64_t K, int64_t ldx, int64_t ldu, int act,
                                                      int pow2, uint8_t* __restrict__ q, int64_t ldq,
                                                      float* __restrict__ scales, int64_t s_ld, int64_t n_groups) {
    const int sub = threadIdx.x & 7;
    for (int64_t i = (int64_t)blockIdx.x * GPB + (threadIdx.x >> 3); i < n_groups; i += (int64_t)gridDim.x * GPB) {
        const int64_t b = i / M, m = i - b * M;
        const int64_t k = b * BLK + 16 * sub;
        const bool in = k < K;  // (K is a multiple of 16)
        float v[16];
        // lanes past the row's end read its first inputs and count as zeros
        load16<T>(x + (m * ldx + (in ? k : 0)) * T::SIZE, v);
        if constexpr (GLU) {
            float w[16];
            load16<T>(u + (m * ldu + (in ? k : 0)) * T::SIZE, w);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = gqd::act_fn(act, v[j]) * w[j];
        }
        if (!in) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
        }
        float s;
        const u32x4 o = quantise(v, pow2, s);
        if (in) *reinterpret_cast<u32x4*>(q + m * ldq + k) = o;
        if (sub == 0) scales[b * s_ld + m] = s;
    }
}

template <typename T, bool GLU>
hipError_t launch(const void* x, const void* u, int64_t M, int64_t K, int64_t ldx, int64_t ldu, int act, int pow2,
                  uint8_t* q, int64_t ldq, float* scales, int64_t s_ld, hipStream_t s) {
    const int64_t groups = M * ((K + BLK - 1) / BLK);
    const int64_t want = (groups + GPB - 1) / GPB;
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : (1 << 20));
    hipLaunchKernelGGL((k_f8_quant<T, GLU>), dim3(grid), dim3(THREADS), 0, s, static_cast<const uint8_t*>(x),
                       static_cast<const uint8_t*>(u), M, K, ldx, ldu, act, pow2, q, ldq, scales, s_ld, groups);
    return hipGetLastError();
}

template <bool GLU>
hipError_t dispatch(const void* x, const void* u, int dtype, int64_t M, int64_t K, int64_t ldx, int64_t ldu, int act,
                    int pow2, uint8_t* q, int64_t ldq, float* scales, int64_t s_ld, hipStream_t s) {
    if (dtype == gqd::DT_F32)
        return launch<f32_t, GLU>(x, u, M, K, ldx, ldu, act, pow2, q, ldq, scales, s_ld, s);
    if (dtype == gqd::DT_BF16)
        return launch<bf16_t, GLU>(x, u, M, K, ldx, ldu, act, pow2, q, ldq, scales, s_ld, s);
    return launch<f16_t, GLU>(x, u, M, K, ldx, ldu, act, pow2, q, ldq, scales, s_ld, s);
}

}  // namespace

hipError_t gqk_f8_quant(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx, int pow2, uint8_t* q,
                        int64_t ldq, float* scales, int64_t s_ld, hipStream_t s) {
    return dispatch<false>(x, nullptr, dtype, M, K, ldx, 0, 0, pow2, q, ldq, scales, s_ld, s);
}

hipError_t gqk_f8_glu_quant(const void* g, const void* u, int dtype, int64_t M, int64_t K, int64_t ldg, int64_t ldu,
                            int act, int pow2, uint8_t* q, int64_t ldq, float* scales, int64_t s_ld, hipStream_t s) {
    return dispatch<true>(g, u, dtype, M, K, ldg, ldu, act, pow2, q, ldq, scales, s_ld, s);
}
