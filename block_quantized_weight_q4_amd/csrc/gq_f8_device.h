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

// Host: a grid dimension counts its threads in 32 bits.
inline bool grid_ok(int64_t groups, int threads) { return groups * threads < ((int64_t)1 << 32); }

typedef __amdgpu_buffer_rsrc_t Rsrc;

// Buffer resource of `bytes` (< 2^31) from base; loads beyond them give zeros.
__device__ __forceinline__ Rsrc make_rsrc(const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t NOWHERE = 0x80000000u;  // an offset beyond every resource
// off (below 2^31) where at < end, otherwise beyond every resource; in
// arithmetic, because a branch would change how many loads are issued.
__device__ __forceinline__ uint32_t within(uint32_t off, int at, int end) {
    return off | ((uint32_t)(end - 1 - at) & NOWHERE);
}

// Stores four neighbouring results of a row (n .. n + 3, those below N) as fp32
// or, rounded to nearest even, as bf16; at once where the row's stride allows.
template <typename T>
__device__ __forceinline__ void store4(T* row, int64_t n, int64_t N, bool vec, f32x4 v) {
    if (vec && n + 4 <= N) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4*>(row + n) = v;
        } else {
            const bf16x2 a = {(__bf16)v[0], (__bf16)v[1]}, b = {(__bf16)v[2], (__bf16)v[3]};
            *reinterpret_cast<u32x2*>(row + n) =
                u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
        }
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (n + r < N) {
            if constexpr (sizeof(T) == 4) row[n + r] = v[r];
            else row[n + r] = gqd::f2bf(v[r]);
        }
}

// Eight neighbouring results: lo, then hi.
template <typename T>
__device__ __forceinline__ void store8(T* row, int64_t n, int64_t N, bool vec, f32x4 lo, f32x4 hi) {
    if constexpr (sizeof(T) == 2) {
        if (vec && n + 8 <= N) {
            const bf16x2 a = {(__bf16)lo[0], (__bf16)lo[1]}, b = {(__bf16)lo[2], (__bf16)lo[3]};
            const bf16x2 c = {(__bf16)hi[0], (__bf16)hi[1]}, d = {(__bf16)hi[2], (__bf16)hi[3]};
            *reinterpret_cast<u32x4*>(row + n) =
                u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                      __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
            return;
        }
    }
    const bool vec4 = sizeof(T) == 4 && vec;
    store4(row, n, N, vec4, lo);
    store4(row, n + 4, N, vec4, hi);
}

__device__ __forceinline__ u32x4 bld16(Rsrc r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// ---- global-to-LDS copies (the loads that write LDS without registers) ----
// Each lane of an instruction brings 16 bytes from an address of its own; they
// land at lds + 16 * lane.  A kernel that uses them waits for them itself.
typedef __attribute__((address_space(3))) void* LdsPtr;
typedef const __attribute__((address_space(1))) void* GlobalPtr;

// (base: the same for the whole wavefront, off + base below 2^31; whether the
// range check counts base is left open: where off is within the resource, off +
// base must be too)
__device__ __forceinline__ void copy16(Rsrc r, uint32_t off, uint8_t* lds, uint32_t base = 0) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)lds, 16, (int)off, (int)base, 0, 0);
}
__device__ __forceinline__ void copy16(const uint8_t* p, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)p, (LdsPtr)lds, 16, 0, 0);
}
// 4 bytes a lane, at lds + 4 * lane.
__device__ __forceinline__ void copy4(const float* p, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)p, (LdsPtr)lds, 4, 0, 0);
}

// Until at most N of this wavefront's loads and copies are outstanding
// (gfx9 encoding: vmcnt in bits 3:0 and 15:14, the other counters at their
// maxima); what reads the copied data stays behind it.
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
// Until this wavefront's LDS reads have returned: what overwrites the LDS that
// they read stays behind it.
__device__ __forceinline__ void wait_reads() {
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (3 << 14));  // lgkmcnt(0)
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Stores a value as fp32 or, rounded to nearest even, as bf16.
template <typename T>
__device__ __forceinline__ void store_as(T* p, float v) {
    if constexpr (sizeof(T) == 4) *p = v;
    else *p = gqd::f2bf(v);
}

}  // namespace gqf8
