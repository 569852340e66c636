// gq_f8_device.h -- device helpers of the block-scaled 8-bit kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_device.h"

namespace gqf8 {

using gqd::f32x4;
using gqd::u32x2;
using gqd::u32x4;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int BLK = 128;  // inputs per activation scale; rows and inputs per weight scale

// One 16 x 16 tile over 128 inputs: lane l holds 32 bytes of row l % 16 of each
// operand (the four lanes of a row split its 128 inputs; both operands in the
// same way, so which lane holds which inputs does not matter) and of the result
// the elements (4 (l / 16) + r, l % 16).
//
// mfma8: the 8-bit matrix instruction.  Measured: it adds the products of eight
// inputs in fixed point, cut off 13 bits below the exponent of the largest of
// them (products of e4m3 values have 8 bits), and those sums in fp32; on
// quantised N(0, 1) rows the result is off by 1.5e-5 of its size, far below the
// 2^-9 of a bf16 result but above what an fp32 result should carry.
__device__ __forceinline__ f32x4 mfma8(i32x8 a, i32x8 b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{}, 0, 0, 0, 0, 0, 0);
}

// Eight e4m3 values as bf16 (exact).
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// mfma16: the same product with both operands widened to bf16, at half the
// rate: exact products, sums in fp32 (measured: bits down to 2^-23 of the
// largest product kept; 1e-8 off on the same rows).
struct Wide {
    bf16x8 v[4];
};
__device__ __forceinline__ Wide widen(i32x8 q) {
    return Wide{{widen(q[0], q[1]), widen(q[2], q[3]), widen(q[4], q[5]), widen(q[6], q[7])}};
}
__device__ __forceinline__ f32x4 mfma16(const Wide& a, const Wide& b) {
    f32x4 d{};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
    return d;
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Stores a value as fp32 or, rounded to nearest even, as bf16.
template <typename T>
__device__ __forceinline__ void store_as(T* p, float v) {
    if constexpr (sizeof(T) == 4) *p = v;
    else *p = gqd::f2bf(v);
}

}  // namespace gqf8
