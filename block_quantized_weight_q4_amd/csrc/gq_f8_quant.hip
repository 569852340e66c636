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
// Bound by HBM: each input is read once and each byte written once; 3015 x 5120
// bf16 take 9.3 us (5.0 TB/s, a 1 GiB copy reaches 5.1), the gated unit of 3015
// x 17408 55.9 us (4.7 TB/s; 60.9 us with expf, tanhf and a division, when the
// vector unit took as long as the memory).  Eight lanes share a group: each holds
// 16 inputs (two or four 16-byte loads, one 16-byte store) and three DPP / xor
// steps give the group's maximum.  The maximum is taken over the magnitudes' bit patterns, where infinities and
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

// 1 / (1 + exp(-z)): exp2 of -z log2(e), whose product's rounding is put back
// into the power (otherwise |z| / 2 steps of it), and the hardware's reciprocal
// (one step).  z is kept where the power is finite; a NaN comes back through
// the factor that the caller multiplies with.
__device__ __forceinline__ float sigmoid(float z) {
    constexpr float L = -1.44269504089f, LN2 = 0.69314718056f;
    z = __builtin_amdgcn_fmed3f(z, -87.0f, 87.0f);
    const float t = z * L, r = __builtin_fmaf(z, L, -t);
    float e = __builtin_amdgcn_exp2f(t);
    e = __builtin_fmaf(e, r * LN2, e);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// act of a gated unit: silu(g) = g sigmoid(g), and the tanh form of gelu as
// g sigmoid(2 sqrt(2 / pi) (g + 0.044715 g^3)), since (1 + tanh v) / 2 = sigmoid(2 v).
__device__ __forceinline__ float act_of(int act, float g) {
    if (act == 0) return g * sigmoid(g);
    return g * sigmoid(1.5957691216f * __builtin_fmaf(0.044715f * g, g * g, g));
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
            const float x = v[4 * j + i], y0 = x * r;
            y[i] = __builtin_fmaf(__builtin_fmaf(-y0, s, x), r, y0);
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
        q[j] = finite ? (uint32_t)w : 0u;
    }
    scale = finite ? s : __builtin_nanf("");
    return q;
}

// A workgroup takes RPB rows by GPB / RPB groups: a wavefront reads 1 KB runs
// of rows, and the scales of neighbouring rows are written side by side.
// (32 rows by one group to 2 by 16: within 2%.)
constexpr int RPB = 8, CPB = GPB / RPB;

template <typename T, bool GLU>
__global__ __launch_bounds__(THREADS) void k_f8_quant(const uint8_t* __restrict__ x, const uint8_t* __restrict__ u,
                                                      int64_t M, int64_t K, int64_t ldx, int64_t ldu, int act,
                                                      int pow2, uint8_t* __restrict__ q, int64_t ldq,
                                                      float* __restrict__ scales, int64_t s_ld) {
    const int sub = threadIdx.x & 7, g = threadIdx.x >> 3;
    const int64_t b = (int64_t)blockIdx.y * CPB + g % CPB;
    const int64_t k = b * BLK + 16 * sub;
    if (b * BLK >= K) return;
    const bool in = k < K;  // (K is a multiple of 16)
    for (int64_t m = (int64_t)blockIdx.x * RPB + g / CPB; m < M; m += (int64_t)gridDim.x * RPB) {
        float v[16];
        // lanes past the row's end read its first inputs and count as zeros
        load16<T>(x + (m * ldx + (in ? k : 0)) * T::SIZE, v);
        if constexpr (GLU) {
            float w[16];
            load16<T>(u + (m * ldu + (in ? k : 0)) * T::SIZE, w);
            if (act == 0) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = act_of(0, v[j]) * w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = act_of(1, v[j]) * w[j];
            }
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
    // (K is at most 2^22: at most 2^15 groups of a row)
    const int64_t gx = (M + RPB - 1) / RPB, gy = (K + BLK * CPB - 1) / (BLK * CPB);
    const dim3 grid((unsigned)(gx < (1 << 20) ? gx : (1 << 20)), (unsigned)gy);
    hipLaunchKernelGGL((k_f8_quant<T, GLU>), grid, dim3(THREADS), 0, s, static_cast<const uint8_t*>(x),
                       static_cast<const uint8_t*>(u), M, K, ldx, ldu, act, pow2, q, ldq, scales, s_ld);
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
