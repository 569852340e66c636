// gq_g4_dx_stream.h -- the gradient of a few rows with respect to the inputs of a
// product with 4-bit weights, bound by the stream of weights (gfx950, wave64).
//
// dX[m][k] = sum_n s[n][k / G] (q[n][k] - z[n][k / G]) dY[m][n]: the scales vary
// along the sum, so each weight is formed first, exactly, and rounded to 16 bits
// for the matrix cores.
//
// A workgroup has 64 columns of W and splits its N rows over its W wavefronts:
// wavefront w takes the blocks of 32 H rows w, w + W, ...  Each has a buffer of LDS
// of its own, which global-to-LDS copies fill with its next block as soon as this
// one's bytes are in registers; the rows of dY, which all workgroups share, come
// from the caches straight into registers.  The partial sums are joined in LDS in
// wavefront order.
//
// 16 rows of 17408 x 5120 (46 MB): 53 us, of 2560 x 9728 13 us; bound by forming the
// weights (about 20 instructions for eight) on as many CUs as there are 64 columns: 80 and
// 152 of 256.  (Tiles, whose wavefronts share a stage, took 139 and 24 us.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_stream.h"
#include "gq_g4_device.h"
#include "gq_g4_internal.h"

namespace gqg4 {

// Weights of rows 2 i and 2 i + 1 of four neighbouring columns, as dword i of the
// operands of those columns: w0, w1 their bytes (two a row), f (512 s, -z s) of the
// two rows.  A nibble as an e4m3 byte is q 2^-9; s (q - z) is exact in fp32.
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

template <int MT, int W, int H>
struct DxStream {
    static constexpr int BM = 16 * MT, BN = 64, BR = 32 * H;
    static constexpr int WB = BR * 32;                // bytes of weights of a wavefront
    static constexpr int SB = 2 * BR * 8;             // its scales: two groups at most
    static constexpr int JOIN = 4 * MT * 1024;
    static constexpr int ONE = WB + SB;
    static constexpr int BYTES = W * (ONE > JOIN ? ONE : JOIN);
    static_assert(BR % 64 == 0, "whole wavefronts of scales");
};

// Rows [0, rows) of dy (1 <= rows <= 16 MT; rows past them repeat the last) by columns
// k0 .. k0 + 63 of W.
template <typename T, int MT, int W, int H>
__device__ __forceinline__ void dx_stream(const G4Weights& wt, const uint16_t* __restrict__ dy, int64_t lddy, int rows,
                                          uint16_t* __restrict__ dx, int64_t lddx, int64_t k0, uint8_t* smem) {
    using S = DxStream<MT, W, H>;
    constexpr int BR = S::BR;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int64_t N = wt.N, K = wt.K, row_bytes = K / 2, KG = (K + wt.group - 1) / wt.group;
    const int NB = (int)((N + BR - 1) / BR);
    uint8_t* mine = smem + wave * S::ONE;
    float* panel = reinterpret_cast<float*>(mine + S::WB);  // [group][row]: 512 s and -z s

    // W: 32 rows of 32 bytes a copy, row 8 a + b at 4 b + a, so that the four rows, 8 apart,
    // that the lanes read at once lie in different banks
    const int at = lane >> 1, cr = 8 * (at & 3) + (at >> 2), chunk = 16 * (lane & 1);
    const uint32_t woff = within((uint32_t)(cr * row_bytes) + chunk, chunk, (int)(K - k0 < 64 ? K - k0 : 64) / 2);
    const int64_t g0 = k0 / wt.group, g1 = wt.group == 32 && g0 + 1 < KG ? g0 + 1 : g0;
    const uint16_t* p[MT];  // this lane's eight columns of dY of a block
#pragma unroll
    for (int j = 0; j < MT; ++j) p[j] = dy + (16 * j + fr < rows ? 16 * j + fr : rows - 1) * lddy + 8 * fq;

    u32x4 b[H][MT];
    uint32_t sc[H / 2][2], zp[H / 2][2];
    auto load = [&](int nb) __attribute__((always_inline)) {
        const int64_t n = (int64_t)nb * BR;
        const int left = n < N ? (int)(N - n < BR ? N - n : BR) : 0;
        const Rsrc wr = make_rsrc(wt.W + (left ? n : 0) * row_bytes + k0 / 2, left ? left * row_bytes - k0 / 2 : 0);
#pragma unroll
        for (int h = 0; h < H; ++h) copy16(wr, woff + (uint32_t)(32 * h * row_bytes), mine + 1024 * h);
#pragma unroll
        for (int h = 0; h < H / 2; ++h) {
            const int64_t r = 64 * h + lane < left ? n + 64 * h + lane : 0;
            sc[h][0] = wt.scales[r * KG + g0];
            sc[h][1] = wt.scales[r * KG + g1];
            zp[h][0] = zp[h][1] = 8;
            if (wt.zeros) {
                zp[h][0] = wt.zeros[r * KG + g0];
                zp[h][1] = wt.zeros[r * KG + g1];
            }
            if (64 * h + lane >= left) sc[h][0] = sc[h][1] = 0;  // (rows past N are zeros)
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
    f32x4 acc[4][MT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[t][j] = f32x4{};
    // lane: columns 4 fr .. + 3 (two bytes), rows 32 h + 8 fq .. + 7
    const int wat = 32 * fq + 2 * fr, gsel = wt.group == 32 ? fr >> 3 : 0;
    if (wave < NB) {
        load(wave);
        for (int nb = wave; nb < NB; nb += W) {
            wait_copies<0>();
            uint32_t w[H][8];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int i = 0; i < 8; ++i) w[h][i] = *reinterpret_cast<const uint16_t*>(mine + 1024 * h + 128 * i + wat);
#pragma unroll
            for (int h = 0; h < H / 2; ++h)
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float f = scale_f32(sc[h][g], wt.s_f16);
                    float* o = panel + g * (2 * BR) + 2 * (64 * h + lane);
                    o[0] = 512.0f * f;
                    o[1] = -(float)(zp[h][g] & 15u) * f;
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
                u32x4 a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) weights_2x4<T>(w[h][2 * i], w[h][2 * i + 1], sp[i], a, i);
#pragma unroll
                for (int t = 0; t < 4; ++t)
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
    f32x4* part = reinterpret_cast<f32x4*>(smem);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            part[(wave * (4 * MT) + 4 * j + r) * 64 + lane] = f32x4{acc[0][j][r], acc[1][j][r], acc[2][j][r], acc[3][j][r]};
    __syncthreads();
    for (int c = wave; c < 4 * MT; c += W) {
        f32x4 v = part[c * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 o = part[(w * (4 * MT) + c) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += o[r];
        }
        // lane: columns 16 fq + 4 (c % 4) .. + 3 of row 16 (c / 4) + fr
        const int64_t k = k0 + 16 * fq + 4 * (c & 3);
        const int row = 16 * (c >> 2) + fr;
        if (row < rows && k < K) {  // (K is a multiple of 32)
            const u32x2 o{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
            __builtin_memcpy(dx + row * lddx + k, &o, 8);
        }
    }
}

}  // namespace gqg4
