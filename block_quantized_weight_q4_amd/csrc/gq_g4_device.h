// gq_g4_device.h -- device helpers of the 4-bit kernels with group scales
// (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_device.h"

namespace gqg4 {

using gqf8::bf16x2;
using gqf8::bf16x8;
using gqf8::bld16;
using gqf8::copy16;
using gqf8::grid_ok;
using gqf8::make_rsrc;
using gqf8::Rsrc;
using gqf8::wait_copies;
using gqf8::wait_reads;
using gqf8::within;
using gqd::f32x4;
using gqd::u32x2;
using gqd::u32x4;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 16-bit element types of the products' inputs.
//
// Weights that are rounded to them are formed as fma(q 2^-9, a, b): a nibble as an e4m3
// byte is q 2^-9 (subnormal below 8, the first normal binade from 8 on), which one
// instruction converts two at a time.  affine() gives a and b of a scale and its zero
// point; the fma is exact in fp32 (16 bits), so the rounding to 16 bits is the only one.
// UNIT: what a sum of such weights is multiplied with.
struct Bf16 {
    typedef bf16x8 x8;
    static constexpr int dtype = gqd::DT_BF16;
    // 2^-9 of the weights: a scale times 512 would be infinite from 2^119 on.  (Weights
    // below 2^-117 are subnormal bf16 numbers so.)
    static constexpr float UNIT = 512.0f;
    static __device__ __forceinline__ gqf8::f32x2 affine(float s, uint32_t z) {
        return gqf8::f32x2{s, (float)z * -0x1p-9f * s};
    }
    static __device__ __forceinline__ uint16_t narrow(float v) { return gqd::f2bf(v); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    }
    static __device__ __forceinline__ f32x4 mfma(x8 a, x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(x8 a, x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
struct F16 {
    typedef f16x8 x8;
    static constexpr int dtype = gqd::DT_F16;
    // The weights themselves: fp16 has no range to spare.  A finite scale above 2^112 becomes
    // that, so that no product overflows: its weights are zeros or infinite either way.
    static constexpr float UNIT = 1.0f;
    static __device__ __forceinline__ gqf8::f32x2 affine(float s, uint32_t z) {
        const float m = __builtin_fabsf(s);
        if (m > 0x1p112f && m < __builtin_inff()) s = __builtin_copysignf(0x1p112f, s);
        return gqf8::f32x2{512.0f * s, -(float)z * s};
    }
    static __device__ __forceinline__ uint16_t narrow(float v) { return gqd::f2h(v); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
    }
    static __device__ __forceinline__ f32x4 mfma(x8 a, x8 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(x8 a, x8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

__device__ __forceinline__ float scale_f32(uint32_t bits16, int s_f16) {
    const float h = gqd::h2f(bits16), b = gqd::bf2f((uint16_t)bits16);
    return s_f16 ? h : b;
}

// Sums of weights in T's unit, as they are.
template <typename T, typename V, int N = sizeof(V) / 4>
__device__ __forceinline__ V in_unit(V v) {
    if constexpr (T::UNIT != 1.0f) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= T::UNIT;
    }
    return v;
}

// Quants minus zero points of a dword's eight nibbles, as signed bytes: even
// inputs in lo, odd ones in hi.  Without zero points (ZP false) the bytes are 16
// (q - 8): the nibble in a byte's upper half with its top bit flipped; UNIT is
// what their scale is multiplied with.  With them the byte 0x80 | q stays
// positive when the zero point (z4: it, in four bytes) is taken off, so that
// nothing is borrowed from a neighbour.
template <bool ZP>
struct Centred {
    static constexpr float UNIT = ZP ? 1.0f : 1.0f / 16;
    uint32_t lo, hi;
    __device__ __forceinline__ Centred(uint32_t w, uint32_t z4) {
        if constexpr (ZP) {
            lo = (((w & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
            hi = ((((w >> 4) & 0x0f0f0f0fu) | 0x80808080u) - z4) ^ 0x80808080u;
        } else {
            lo = ((w << 4) & 0xf0f0f0f0u) ^ 0x80808080u;
            hi = (w & 0xf0f0f0f0u) ^ 0x80808080u;
        }
    }
    // input i of the eight
    __device__ __forceinline__ float at(int i) const {
        return (float)(int)(int8_t)((i & 1 ? hi : lo) >> (8 * (i >> 1)));
    }
};

// Zero points of a group, in four bytes.
__device__ __forceinline__ uint32_t zero4(uint32_t z) { return (z & 15u) * 0x01010101u; }

// The eight as an operand of the matrix instructions (exact: at most 8 bits).
template <typename T, bool ZP>
__device__ __forceinline__ typename T::x8 operand(uint32_t w, uint32_t z4) {
    const Centred<ZP> c(w, z4);
    return __builtin_bit_cast(typename T::x8, u32x4{T::pack(c.at(0), c.at(1)), T::pack(c.at(2), c.at(3)),
                                                   T::pack(c.at(4), c.at(5)), T::pack(c.at(6), c.at(7))});
}

// Stores a value as the type that dtype says.
__device__ __forceinline__ void store_as(void* p, int64_t i, int dtype, float v) {
    if (dtype == gqd::DT_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = dtype == gqd::DT_BF16 ? gqd::f2bf(v) : gqd::f2h(v);
}
// The first c of four neighbours (of any alignment).
__device__ __forceinline__ void store_as(void* p, int64_t i, int dtype, f32x4 v, int c) {
    if (c < 4) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < c) store_as(p, i + e, dtype, v[e]);
    } else if (dtype == gqd::DT_F32) {
        __builtin_memcpy(static_cast<float*>(p) + i, &v, 16);
    } else {
        const u32x2 o = dtype == gqd::DT_BF16 ? u32x2{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3])}
                                              : u32x2{F16::pack(v[0], v[1]), F16::pack(v[2], v[3])};
        __builtin_memcpy(static_cast<uint16_t*>(p) + i, &o, 8);
    }
}

}  // namespace gqg4
