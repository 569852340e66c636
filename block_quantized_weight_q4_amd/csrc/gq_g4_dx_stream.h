// gq_g4_dx_stream.h -- the gradient of a few rows with respect to the inputs of a
// product with 4-bit weights, bound by the stream of weights (gfx950, wave64).
//
// dX[m][k] = sum_n s[n][k / G] (q[n][k] - z[n][k / G]) dY[m][n]: the scales vary
// along the sum, so each weight is formed first, exactly, and rounded to 16 bits
// for the matrix cores.
//
// A workgroup has 64 or 32 columns of W and splits its N rows over its W wavefronts:
// wavefront w takes the blocks of 32 H rows w, w + W, ...  Each has a buffer of LDS
// of its own, which global-to-LDS copies fill with its next block as soon as this
// one's bytes are in registers; the rows of dY, which all workgroups share, come
// from the caches straight into registers.  The partial sums are joined in LDS in
// wavefront order.
//
// 16 rows of 17408 x 5120 (46 MB): 44 us, of 2560 x 9728 12.5 us; bound by forming the
// weights (about 20 instructions for eight) on as many CUs as there are 32 or 64 columns:
// 160 and 152 of 256.  (Tiles, whose wavefronts share a stage, took 139 and 24 us.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_stream.h"
#include "gq_g4_device.h"
#include "gq_g4_internal.h"

namespace gqg4 {

// Weights of rows 2 i and 2 i + 1 of four neighbouring columns, as dword i of the
// operands of those columns, in T's unit: w0, w1 their bytes (two a row), f (T::affine)
// of the two rows.
template <typename T>
__device__ __forceinline__ void weights_2x4(uint32_t w0, uint32_t w1, f32x4 f, u32x4 (&a)[4], int i) {
    // (joined by a byte permute: a read into the upper half of a register waits for the lower one's)
    const uint32_t v = __builtin_amdgcn_perm(w1, w0, 0x05040100u);
    const int lo = (int)(v & 0x0f0f0f0fu), hi = (int)((v >> 4) & 0x0f0f0f0fu);
    const gqf8::f32x2 e0 = __builtin_amdgcn_cvt_pk_f32_fp8(lo, false);
    const gqf8::f32x2 e1 = __builtin_amdgcn_cvt_pk_f32_fp8(lo, true);
    const gqf8::f32x2 o0 = __builtin_amdgcn_cvt_pk_f32_fp8(hi, false);
    const gqf8::f32x2 o1 = __builtin_amdgcn_cvt_pk_f32_fp8(hi, true);
    auto f0 = [&](float q) { return __builtin_fmaf(q, f[0], f[1]); };
    auto f1 = [&](float q) { return __builtin_fmaf(q, f[2], f[3]); };
    a[0][i] = T::pack(f0(e0.x), f1(e1.x));
    a[1][i] = T::pack(f0(o0.x), f1(o1.x));
    a[2][i] = T::pack(f0(e0.y), f1(e1.y));
    a[3][i] = T::pack(f0(o0.y), f1(o1.y));
}

// Of two neighbouring columns and rows 4 k .. + 3: w0 to w3 their bytes (one a row), f
// and g the scales of rows 4 k, 4 k + 1 and of the other two.
template <typename T>
__device__ __forceinline__ void weights_4x2(const uint32_t* w, f32x4 f, f32x4 g, u32x4 (&a)[2], int k) {
    const uint32_t v = __builtin_amdgcn_perm(__builtin_amdgcn_perm(w[3], w[2], 0x0c0c0400u),
                                             __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u), 0x05040100u);
    const uint32_t q[2] = {v & 0x0f0f0f0fu, (v >> 4) & 0x0f0f0f0fu};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const gqf8::f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[t], false);
        const gqf8::f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[t], true);
        a[t][2 * k] = T::pack(__builtin_fmaf(b.x, f[0], f[1]), __builtin_fmaf(b.y, f[2], f[3]));
        a[t][2 * k + 1] = T::pack(__builtin_fmaf(c.x, g[0], g[1]), __builtin_fmaf(c.y, g[2], g[3]));
    }
}

// C columns (64 or 32), of C / 16 operands.
template <int MT, int W, int H, int C>
struct DxStream {
    static constexpr int BM = 16 * MT, BN = C, BR = 32 * H, NT = C / 16;
    static constexpr int GROUPS = C / 32;             // groups of the columns, at most
    static constexpr int WB = BR * (C / 2);           // bytes of weights of a wavefront
    static constexpr int SB = GROUPS * BR * 8;        // its scales
    static constexpr int JOIN = NT * MT * 1024;
    static constexpr int ONE = WB + SB;
    static constexpr int BYTES = W * (ONE > JOIN ? ONE : JOIN);
    static_assert(BR % 64 == 0 && (C == 64 || C == 32), "whole wavefronts of scales");
};

// Rows [0, rows) of dy (1 <= rows <= 16 MT; rows past them repeat the last) by columns
// k0 .. k0 + C - 1 of W.
template <typename T, int MT, int W, int H, int C>
__device__ __forceinline__ void dx_stream(const G4Weights& wt, const uint16_t* __restrict__ dy, int64_t lddy, int rows,
                                          uint16_t* __restrict__ dx, int64_t lddx, int64_t k0, uint8_t* smem) {
    using S = DxStream<MT, W, H, C>;
    constexpr int BR = S::BR, NT = S::NT, GROUPS = S::GROUPS;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int64_t N = wt.N, K = wt.K, row_bytes = K / 2, KG = (K + wt.group - 1) / wt.group;
    const int NB = (int)((N + BR - 1) / BR);
    uint8_t* mine = smem + wave * S::ONE;
    float* panel = reinterpret_cast<float*>(mine + S::WB);  // [group][row]: T::affine

    // W: C / 2 bytes of 32 rows (64 of 32 columns) a copy, row 8 a + b of 32 at 4 b + a, so that
    // the four rows, 8 apart, that the lanes read at once lie in different banks
    constexpr int COPY = 2048 / C, CHUNKS = C / 32;  // rows of a copy, 16-byte chunks of a row
    const int at = lane / CHUNKS, cr = (at & 32) + 8 * (at & 3) + ((at >> 2) & 7), chunk = 16 * (lane % CHUNKS);
    const uint32_t woff = within((uint32_t)(cr * row_bytes) + chunk, chunk, (int)(K - k0 < C ? K - k0 : C) / 2);
    const int64_t g0 = k0 / wt.group, g1 = wt.group == 32 && g0 + 1 < KG ? g0 + 1 : g0;
    const uint16_t* p[MT];  // this lane's eight columns of dY of a block
#pragma unroll
    for (int j = 0; j < MT; ++j) p[j] = dy + (16 * j + fr < rows ? 16 * j + fr : rows - 1) * lddy + 8 * fq;

    u32x4 b[H][MT];
    uint32_t sc[H / 2][GROUPS], zp[H / 2][GROUPS];
    auto load = [&](int nb) __attribute__((always_inline)) {
        const int64_t n = (int64_t)nb * BR;
        const int left = n < N ? (int)(N - n < BR ? N - n : BR) : 0;
        const Rsrc wr = make_rsrc(wt.W + (left ? n : 0) * row_bytes + k0 / 2, left ? left * row_bytes - k0 / 2 : 0);
#pragma unroll
        for (int h = 0; h < BR / COPY; ++h) copy16(wr, woff + (uint32_t)(COPY * h * row_bytes), mine + 1024 * h);
#pragma unroll
        for (int h = 0; h < H / 2; ++h) {
            const int64_t r = 64 * h + lane < left ? n + 64 * h + lane : 0;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                sc[h][g] = wt.scales[r * KG + (g ? g1 : g0)];
                zp[h][g] = 8;
            }
            if (wt.zeros) {
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) zp[h][g] = wt.zeros[r * KG + (g ? g1 : g0)];
            }
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
                if (64 * h + lane >= left) sc[h][g] = 0;  // (rows past N are zeros)
        }
        if (left == BR) {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < MT; ++j) __builtin_memcpy(&b[h][j], p[j] + n + 32 * h, 16);  // (of any alignment)
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const int c = left - (32 * h + 8 * fq);  // columns that there are
                    u32x4 v{};
                    if (c >= 8) {
                        __builtin_memcpy(&v, p[j] + n + 32 * h, 16);
                    } else {
#pragma unroll
                        for (int i = 0; i < 7; ++i)
                            if (i < c) v[i / 2] |= (uint32_t)p[j][n + 32 * h + i] << (16 * (i & 1));
                    }
                    __asm__ volatile("" : "+v"(v) : : "memory");  // (one piece at a time, for the registers' sake)
                    b[h][j] = v;
                }
        }
    };
    f32x4 acc[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[t][j] = f32x4{};
    // lane: columns NT fr .. (two bytes, or one), rows 32 h + 8 fq .. + 7
    const int wat = (C / 2) * fq + (C / 32) * fr, gsel = GROUPS == 2 && wt.group == 32 ? fr >> 3 : 0;
    if (wave < NB) {
        load(wave);
        for (int nb = wave; nb < NB; nb += W) {
            wait_copies<0>();
            uint32_t w[H][8];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint8_t* q = mine + (16 * C) * h + (2 * C) * i + wat;
                    if constexpr (C == 64) w[h][i] = *reinterpret_cast<const uint16_t*>(q);
                    else w[h][i] = *q;
                }
#pragma unroll
            for (int h = 0; h < H / 2; ++h)
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    const float f = scale_f32(sc[h][g], wt.s_f16);
                    const gqf8::f32x2 v = T::affine(f, zp[h][g] & 15u);
                    float* o = panel + g * (2 * BR) + 2 * (64 * h + lane);
                    o[0] = v.x;
                    o[1] = v.y;
                }
            u32x4 x[H][MT];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int j = 0; j < MT; ++j) x[h][j] = b[h][j];
            wait_reads();
            load(nb + W);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const f32x4* sp = reinterpret_cast<const f32x4*>(panel + gsel * (2 * BR) + 2 * (32 * h + 8 * fq));
                u32x4 a[NT];
                if constexpr (C == 64) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) weights_2x4<T>(w[h][2 * i], w[h][2 * i + 1], sp[i], a, i);
                } else {
#pragma unroll
                    for (int k = 0; k < 2; ++k) weights_4x2<T>(&w[h][4 * k], sp[2 * k], sp[2 * k + 1], a, k);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[t][j] = T::mfma(__builtin_bit_cast(typename T::x8, a[t]),
                                            __builtin_bit_cast(typename T::x8, x[h][j]), acc[t][j]);
            }
        }
    }
    wait_copies<0>();
    __syncthreads();
    // the join: partial sums of every wavefront, added in their order
    constexpr int FOURS = NT * MT;  // of a lane: four neighbouring columns each
    f32x4* part = reinterpret_cast<f32x4*>(smem);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            f32x4 v;
            if constexpr (C == 64) v = f32x4{acc[0][j][r], acc[1][j][r], acc[2][j][r], acc[3][j][r]};
            else v = f32x4{acc[0][j][2 * r], acc[1][j][2 * r], acc[0][j][2 * r + 1], acc[1][j][2 * r + 1]};
            part[(wave * FOURS + NT * j + r) * 64 + lane] = v;
        }
    __syncthreads();
    for (int c = wave; c < FOURS; c += W) {
        f32x4 v = part[c * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 o = part[(w * FOURS + c) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += o[r];
        }
        // lane: columns 4 NT fq + 4 (c % NT) .. + 3 of row 16 (c / NT) + fr
        const int64_t k = k0 + 4 * NT * fq + 4 * (c % NT);
        const int row = 16 * (c / NT) + fr;
        if (row < rows && k < K) {  // (K is a multiple of 32)
            v = in_unit<T>(v);
            const u32x2 o{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
            __builtin_memcpy(dx + row * lddx + k, &o, 8);
        }
    }
}

}  // namespace gqg4
