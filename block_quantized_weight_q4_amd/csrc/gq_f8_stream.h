// gq_f8_stream.h -- the product of a few rows with block-scaled e4m3 weights,
// bound by the stream of weights (gfx950, wave64): decode vectors, small
// prompts and the experts of a few tokens.
//
// A workgroup owns 16 NT rows of weights and 16 MT rows of X and splits K over
// its W wavefronts: wavefront w takes the 128-input blocks w, w + W, ..., so
// that together they read neighbouring parts of the same rows.  Weights and X
// go through LDS, each wavefront's through a buffer of its own, filled with its
// next block by global-to-LDS copies as soon as the operands are in registers,
// with no barrier before the end (two blocks ahead hold too few wavefronts a CU:
// 19456 x 2560, 8 vectors 12.0 against 10.2 us).  Not because
// anything is shared: a matrix-core operand wants 16 bytes of 16 different
// rows in neighbouring lanes, and loads in that order reach about one lane a
// cycle (measured: 14 bytes a cycle and CU, 33-56 us for 5120 x 17408 and 16
// vectors), whereas a copy brings eight whole 128-byte runs at once and LDS
// serves any order.  The partial sums are joined in LDS in wavefront order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_device.h"

namespace gqf8 {

// How X is given: e4m3 rows with scales, or bf16 / fp32 vectors.
enum { X_E4M3 = 0, X_BF16 = 1, X_F32 = 2 };

// 16-byte position of chunk c of a 128-byte (8 chunks), 256-byte or 512-byte
// row r in LDS: 16 rows at one chunk then cover all banks.
__device__ __forceinline__ int pos128(int r, int c) { return r * 8 + (c ^ ((r >> 1) & 7)); }
__device__ __forceinline__ int pos_wide(int r, int c, int chunks) { return r * chunks + (c ^ (r & 15)); }

// What an fp32 value's upper 16 bits leave of it.
__device__ __forceinline__ uint32_t minus_upper(uint32_t u) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u) - __builtin_bit_cast(float, u & 0xffff0000u));
}

// Eight fp32 values as three bf16 operands whose sum they are: the upper 16
// bits, those of what is left, and the rest (8 + 8 + 8 bits of the mantissa:
// exact while the last is a normal number).
__device__ __forceinline__ void split8(const u32x4& p, const u32x4& q, bf16x8 (&x)[3]) {
    u32x4 part[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u0 = i < 2 ? p[2 * i] : q[2 * i - 4], u1 = i < 2 ? p[2 * i + 1] : q[2 * i - 3];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            part[c][i] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);  // the upper halves of both
            u0 = minus_upper(u0);
            u1 = minus_upper(u1);
        }
    }
#pragma unroll
    for (int c = 0; c < 3; ++c) x[c] = __builtin_bit_cast(bf16x8, part[c]);
}

// Sizes of one block of one wavefront.  XR: rows of X held (a vector product
// of at most XR vectors; columns past them repeat and are not stored).
template <int MT, int NT, int XM, int XR>
struct Stream {
    static constexpr int WI = 2 * NT;                                         // copies of weights
    static constexpr int ROW = XM == X_E4M3 ? 128 : XM == X_BF16 ? 256 : 512; // bytes of a row of X
    static constexpr int XI = XR * ROW / 1024;                                // copies of X
    static constexpr int SCALES = 1024 * (WI + XI);                           // 64 fp32: of X's rows, the last of W
    static constexpr int BYTES = SCALES + 256;
    // fp32 vectors, eight at most: each value is split once, by one lane, and
    // passed on through LDS (sixteen fill all the operand's columns anyway)
    static constexpr bool SHARE = XM == X_F32 && XR <= 8;
    static constexpr int PARTS = SHARE ? 3 * XR * 256 : 0;
    static_assert(XR * ROW % 1024 == 0 && XR <= 16 * MT && MT <= 3, "whole copies, one of scales");
};

// x_row(i): row of X that row i of the tile stands for, any valid
// one past the tile's rows; y_row(i): address of the output row (i < rows).
// smem: W * (BYTES + PARTS) bytes, at least W * NT * MT KB.
template <int MT, int NT, int W, int XM, int XR, typename TY, typename XRow, typename YRow>
__device__ __forceinline__ void stream_tile(const uint8_t* __restrict__ Wt, const float* __restrict__ wsc, int64_t n0,
                                            int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                            const float* __restrict__ xs, int64_t x_stride, int64_t xs_ld, int rows,
                                            bool vec, XRow x_row, YRow y_row, uint8_t* smem) {
    using S = Stream<MT, NT, XM, XR>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int KB = (int)((K + BLK - 1) / BLK);
    const int64_t w_rows = N - n0 < 16 * NT ? N - n0 : 16 * NT;
    const Rsrc wr = make_rsrc(Wt + n0 * K, w_rows * K);
    const float* wsb = wsc + (n0 / BLK) * KB;  // (16 NT rows lie in one block of 128)
    uint8_t* mine = smem + wave * (S::BYTES + S::PARTS);

    // copies: lane's row and 16-byte chunk of each instruction.  What lies past
    // K is read as zeros from W (beyond the resource), and from X as the row's
    // first chunk, which those zeros multiply.
    const int wrow = lane >> 3;
    uint32_t woff[S::WI];
    int wchunk[2];  // (the swizzle has a period of 16 rows: two instructions)
#pragma unroll
    for (int t = 0; t < S::WI; ++t) {
        const int r = 8 * t + wrow;
        wchunk[t & 1] = 16 * ((lane & 7) ^ ((r >> 1) & 7));
        woff[t] = (uint32_t)(r * K + wchunk[t & 1]);
    }
    constexpr int CH = S::ROW / 16, RPI = 64 / CH;  // chunks of a row of X, rows of an instruction
    const uint8_t* xp[S::XI];
    int xchunk[S::XI];
#pragma unroll
    for (int t = 0; t < S::XI; ++t) {
        const int r = RPI * t + lane / CH, c = lane % CH;
        xchunk[t] = 16 * (XM == X_E4M3 ? c ^ ((r >> 1) & 7) : c ^ (r & 15));
        xp[t] = X + (int64_t)x_row(r) * x_stride;
    }
    // scales come the same way: lane i < 16 MT that of row i, the others W's
    const bool xlane = XM == X_E4M3 && lane < 16 * MT;
    const float* sp = xlane ? xs + x_row(lane) : wsb;
    const int64_t sstep = xlane ? xs_ld : 1;
    constexpr int XB = S::ROW / 128;           // bytes of X per input
    const int64_t xbytes = K * XB;
    auto load = [&](int kb) {
        const int kc = kb < KB ? kb : KB - 1;
        uint8_t* d = mine;
        const int64_t k = (int64_t)kb * BLK;
        const int left = k < K ? (int)(K - k) : 0;
#pragma unroll
        for (int t = 0; t < S::WI; ++t)
            copy16(wr, within(woff[t], wchunk[t & 1], left), d + 1024 * t, (uint32_t)k);
#pragma unroll
        for (int t = 0; t < S::XI; ++t)
            copy16(xp[t] + (k * XB + xchunk[t] < xbytes ? k * XB + xchunk[t] : 0), d + 1024 * (S::WI + t));
        copy4(sp + kc * sstep, d + S::SCALES);
    };
    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{};

    // one block: operands from LDS, the next one's copies, the products
    auto step = [&](int kb) {
        const u32x4* d = reinterpret_cast<const u32x4*>(mine);
        u32x4 a[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a[i][h] = d[pos128(16 * i + fr, 4 * h + fq)];
        const u32x4* xd = d + 64 * S::WI;
        const float* sc = reinterpret_cast<const float*>(mine + S::SCALES);
        const float s_w = sc[63];
        float s_x[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) s_x[j] = XM == X_E4M3 ? sc[16 * j + fr] : 1.0f;
        f32x4 p[NT][MT];
        if constexpr (XM == X_E4M3) {
            u32x4 x[MT][2];
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) x[j][h] = xd[pos128(16 * j + fr, 4 * h + fq)];
            wait_reads();
            load(kb + W);
            if constexpr (sizeof(TY) == 4) {
                Wide xw[MT];
#pragma unroll
                for (int j = 0; j < MT; ++j) xw[j] = widen(join(x[j][0], x[j][1]));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const Wide aw = widen(join(a[i][0], a[i][1]));
#pragma unroll
                    for (int j = 0; j < MT; ++j) p[i][j] = mfma16(aw, xw[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        p[i][j] = mfma8(join(a[i][0], a[i][1]), join(x[j][0], x[j][1]));
            }
        } else {
            // chunk c = 4 h + q of the weights meets inputs 16 c .. 16 c + 15 of the vectors
            constexpr int PER = XM == X_BF16 ? 2 : 4;  // 16-byte pieces of them
            constexpr int PARTS = XM == X_BF16 ? 1 : 3;
            const int xr = fr & (XR - 1);
            bf16x8 v[2][2][PARTS];
            if constexpr (S::SHARE) {
                // eight inputs a lane and turn; their three parts at [part][row][eight]
                bf16x8* parts = reinterpret_cast<bf16x8*>(mine + S::BYTES);
#pragma unroll
                for (int u = 0; u < XR / 4; ++u) {
                    const int row = 4 * u + (lane >> 4), o = lane & 15;
                    bf16x8 y[3];
                    split8(xd[pos_wide(row, 2 * o, CH)], xd[pos_wide(row, 2 * o + 1, CH)], y);
#pragma unroll
                    for (int e = 0; e < 3; ++e) parts[pos_wide(e * XR + row, o, 16)] = y[e];
                }
                wait_reads();
                load(kb + W);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 3; ++e) v[h][c][e] = parts[pos_wide(e * XR + xr, 2 * (4 * h + fq) + c, 16)];
            } else {
                u32x4 x[2][PER];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < PER; ++c) x[h][c] = xd[pos_wide(xr, PER * (4 * h + fq) + c, CH)];
                wait_reads();
                load(kb + W);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if constexpr (XM == X_BF16) v[h][c][0] = __builtin_bit_cast(bf16x8, x[h][c]);
                        else split8(x[h][2 * c], x[h][2 * c + 1], v[h][c]);
                    }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                p[i][0] = f32x4{};
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const bf16x8 w = widen((int)a[i][h][2 * c], (int)a[i][h][2 * c + 1]);
#pragma unroll
                        for (int e = PARTS - 1; e >= 0; --e)
                            p[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, v[h][c][e], p[i][0], 0, 0, 0);
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const float f = s_w * s_x[j];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(f, p[i][j][r], acc[i][j][r]);
        }
    };
    if (wave < KB) {
        load(wave);
        for (int kb = wave; kb < KB; kb += W) {
            wait_copies<0>();
            step(kb);
        }
    }
    wait_copies<0>();
    __syncthreads();
    // the join: partial sums of every wavefront, added in their order
    constexpr int TILES = NT * MT;
    f32x4* part = reinterpret_cast<f32x4*>(smem);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) part[(wave * TILES + i * MT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int c = wave; c < TILES; c += W) {
        f32x4 v = part[c * 64 + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 o = part[(w * TILES + c) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += o[r];
        }
        // lane: columns 16 i + 4 q .. + 3 of tile row 16 j + l % 16
        const int i = c / MT, j = c % MT, row = 16 * j + fr;
        if (row < rows) store4(y_row(row), n0 + 16 * i + 4 * fq, N, vec, v);
    }
}

}  // namespace gqf8
