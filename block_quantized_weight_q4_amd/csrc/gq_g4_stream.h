// gq_g4_stream.h -- the product of a few rows of X with 4-bit weights, bound by the
// stream of weights (gfx950, wave64): decode vectors, short prompts, and the few
// rows that each of many experts has.
//
// y[m][n] = sum over groups g of s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) x[m][k]:
// the inner sums are matrix instructions on exact integers, scaled into the fp32
// accumulators group by group.
//
// A workgroup owns 16 NT rows of weights and splits K over its W wavefronts:
// wavefront w takes the 256-input blocks w, w + W, ... (128 bytes a row), so
// that together they read neighbouring parts of the same rows.  Weights and X go
// through LDS, each wavefront's through a buffer of its own that global-to-LDS
// copies fill with its next block as soon as the operands are in registers: a
// copy brings whole 128-byte runs, and LDS gives them out in the order of the
// operands (row l % 16 in lane l).  The partial sums are joined in LDS in
// wavefront order.
//
// 5120 x 17408 with 16 bf16 vectors (49 MB): 20.8 us, 26.9 from HBM alone; 160 workgroups
// on 256 CUs, each with one block in flight a wavefront.  64 rows of 128 experts, 704 x
// 2816 (52 MB): 15.3 us.  Many rows, for fp32 results: 1024 x 17408 x 5120 in 402 us (450
// TFLOP/s), bound by expanding the weights again for every 32 rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_stream.h"
#include "gq_g4_device.h"

namespace gqg4 {

constexpr int BLK = 256;  // inputs of a block

// How X is given.
struct XBf16 : Bf16 {
    static constexpr int SIZE = 2;
};
struct XF16 : F16 {
    static constexpr int SIZE = 2;
};
struct XF32 : Bf16 {  // three bf16 parts
    static constexpr int SIZE = 4;
};

// Bytes of LDS of one wavefront: its weights, its XR rows of X.
template <typename X, int NT, int XR>
struct StreamSize {
    static constexpr int WI = 2 * NT;                  // copies (1 KB) of weights
    static constexpr int ROW = BLK * X::SIZE;          // bytes of a row of X
    static constexpr int XI = XR * ROW / 1024;         // copies of X
    // fp32 rows, eight at most: each value is split once, by one lane, and passed on
    // through LDS (sixteen fill all the operand's columns anyway)
    static constexpr bool SHARE = X::SIZE == 4 && XR <= 8;
    static constexpr int PARTS_AT = 1024 * (WI + XI);
    static constexpr int BYTES = PARTS_AT + (SHARE ? 3 * XR * 512 : 0);
    static constexpr int MT = XR > 16 ? XR / 16 : 1;   // operands of rows of X
    static constexpr int JOIN_ROW = 20;  // floats: a tile's 16 and a gap, so that rows 4 apart lie in other banks
    static constexpr int JOIN = 64 * JOIN_ROW * NT * MT;
    static_assert(XR * ROW % 1024 == 0, "whole copies");
};

// Rows [row0, row0 + rows) of X (1 <= rows <= XR; rows past them repeat the
// last), the 16 NT rows of W from n0.  smem: W * max(BYTES, JOIN) bytes.
// store(i, n, v, c): elements n .. n + c - 1 of row i < rows (1 <= c <= 4).
template <typename X, bool ZP, int G, int NT, int W, int XR, typename Store>
__device__ __forceinline__ void stream_tile(const G4Weights& wt, int64_t n0, const void* __restrict__ Xp,
                                            int64_t ldx, int rows, uint8_t* smem, Store store) {
    using S = StreamSize<X, NT, XR>;
    constexpr int GPB = BLK / G;                // groups of a block
    constexpr int MPG = G / 32;                 // matrix instructions of a group (dwords of a lane)
    constexpr int CH = S::ROW / 16;             // 16-byte chunks of a row of X
    constexpr int MT = S::MT;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int64_t N = wt.N, K = wt.K, row_bytes = K / 2;
    const int KB = (int)((K + BLK - 1) / BLK), KG = (int)((K + G - 1) / G);
    const int64_t w_rows = N - n0 < 16 * NT ? N - n0 : 16 * NT;
    const Rsrc wr = make_rsrc(wt.W + n0 * row_bytes, w_rows * row_bytes);
    const Rsrc xr = make_rsrc(Xp, ((rows - 1) * ldx + K) * X::SIZE);
    uint8_t* mine = smem + wave * S::BYTES;

    // copies: lane's row and 16-byte chunk of each instruction.  What lies past K
    // is read as zeros (beyond the resource) from X; from W too, where they are
    // no zero weights, but meet X's zeros.
    uint32_t woff[S::WI];
    int wchunk[2];  // (the swizzle has a period of 16 rows: two instructions)
#pragma unroll
    for (int t = 0; t < S::WI; ++t) {
        const int r = 8 * t + (lane >> 3);
        wchunk[t & 1] = 16 * ((lane & 7) ^ ((r >> 1) & 7));
        woff[t] = (uint32_t)(r * row_bytes + wchunk[t & 1]);
    }
    uint32_t xoff[S::XI];
    int xchunk[S::XI];
#pragma unroll
    for (int t = 0; t < S::XI; ++t) {
        const int at = 64 * t + lane, r = at / CH, c = at % CH;
        xchunk[t] = 16 * (c ^ (r & 15));
        xoff[t] = (uint32_t)((r < rows ? r : rows - 1) * ldx * X::SIZE) + xchunk[t];
    }
    // scales and zero points of this lane's row of each tile; past the last group zeros
    int64_t srow[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t n = n0 + 16 * i + fr;
        srow[i] = (n < N ? n : N - 1) * KG;
    }
    uint32_t sc[NT][(GPB + 1) / 2], zp[NT][(GPB + 3) / 4];  // of the block that is on its way
    auto load = [&](int kb) {
        const int64_t k = (int64_t)kb * BLK;
        const int wleft = k < K ? (int)(row_bytes - k / 2) : 0;
        const int64_t xleft = k < K ? (K - k) * X::SIZE : 0;
#pragma unroll
        for (int t = 0; t < S::WI; ++t)
            copy16(wr, within(woff[t], wchunk[t & 1], wleft), mine + 1024 * t, (uint32_t)(k / 2));
#pragma unroll
        for (int t = 0; t < S::XI; ++t)
            copy16(xr, within(xoff[t], xchunk[t], (int)(xleft < 4096 ? xleft : 4096)), mine + 1024 * (S::WI + t),
                   (uint32_t)(k * X::SIZE));
        const int g0 = kb * GPB;
        if (g0 + GPB <= KG) {  // (the same for the whole workgroup's rows)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                __builtin_memcpy(sc[i], wt.scales + srow[i] + g0, 2 * GPB);
                if constexpr (ZP) __builtin_memcpy(zp[i], wt.zeros + srow[i] + g0, GPB);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int g = 0; g < GPB; ++g) {
                    const bool in = g0 + g < KG;
                    const uint32_t s = in ? wt.scales[srow[i] + g0 + g] : 0u;
                    sc[i][g / 2] = g & 1 ? sc[i][g / 2] | s << 16 : s;
                    if constexpr (ZP) {
                        const uint32_t z = in ? wt.zeros[srow[i] + g0 + g] : 0u;
                        zp[i][g / 4] = g & 3 ? zp[i][g / 4] | z << (8 * (g & 3)) : z;
                    }
                }
            }
        }
    };
    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{};

    // one block: operands from LDS, the next one's copies, the products
    constexpr int PARTS = X::SIZE == 4 ? 3 : 1;
    const int xrow = XR < 16 ? fr & (XR - 1) : fr;
    auto step = [&](int kb) {
        // group g: MPG dwords of this lane's row, from byte (G / 2) g + 4 MPG fq
        uint32_t a[NT][GPB][MPG];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                const int at = g * (G / 2) + 4 * MPG * fq;  // byte of the row
                const uint8_t* p = mine + 16 * gqf8::pos128(16 * i + fr, at >> 4) + (at & 15);
                __builtin_memcpy(a[i][g], __builtin_assume_aligned(p, 4 * MPG), 4 * MPG);
            }
        const u32x4* xd = reinterpret_cast<const u32x4*>(mine + 1024 * S::WI);
        // (eight inputs g, m: which of the block's)
        auto eight = [&](int g, int m) { return g * (G / 8) + MPG * fq + m; };
        constexpr int PIECES = X::SIZE / 2;  // 16-byte pieces of eight inputs
        u32x4 raw[MT][GPB][MPG][S::SHARE ? 1 : PIECES];
        bf16x8* parts = reinterpret_cast<bf16x8*>(mine + S::PARTS_AT);  // [part][row][eight]
        if constexpr (S::SHARE) {
#pragma unroll
            for (int u = 0; u < (XR * 32 + 63) / 64; ++u) {
                const int at = 64 * u + lane, row = at >> 5, o = at & 31;
                if (XR * 32 >= 64 || lane < XR * 32) {
                    bf16x8 y[3];
                    gqf8::split8(xd[gqf8::pos_wide(row, 2 * o, CH)], xd[gqf8::pos_wide(row, 2 * o + 1, CH)], y);
#pragma unroll
                    for (int e = 0; e < 3; ++e) parts[gqf8::pos_wide(e * XR + row, o, 32)] = y[e];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int g = 0; g < GPB; ++g)
#pragma unroll
                    for (int m = 0; m < MPG; ++m)
#pragma unroll
                        for (int c = 0; c < PIECES; ++c)
                            raw[j][g][m][c] = xd[gqf8::pos_wide(16 * j + xrow, PIECES * eight(g, m) + c, CH)];
        }
        float s[NT][GPB];
        uint32_t z4[NT][GPB];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int g = 0; g < GPB; ++g) {
                s[i][g] = scale_f32(sc[i][g / 2] >> (16 * (g & 1)) & 0xffffu, wt.s_f16) * Centred<ZP>::UNIT;
                z4[i][g] = ZP ? zero4(zp[i][g / 4] >> (8 * (g & 3))) : 0u;
            }
        wait_reads();
        load(kb + W);
#pragma unroll
        for (int g = 0; g < GPB; ++g) {
            typename X::x8 v[MT][MPG][PARTS];
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int m = 0; m < MPG; ++m) {
                    if constexpr (S::SHARE) {
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            v[j][m][e] = parts[gqf8::pos_wide(e * XR + xrow, eight(g, m), 32)];
                    } else if constexpr (PARTS == 3) gqf8::split8(raw[j][g][m][0], raw[j][g][m][1], v[j][m]);
                    else v[j][m][0] = __builtin_bit_cast(typename X::x8, raw[j][g][m][0]);
                }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                f32x4 p[MT];
#pragma unroll
                for (int j = 0; j < MT; ++j) p[j] = f32x4{};
#pragma unroll
                for (int m = 0; m < MPG; ++m) {
                    const typename X::x8 b = operand<X, ZP>(a[i][g][m], z4[i][g]);
#pragma unroll
                    for (int j = 0; j < MT; ++j)
#pragma unroll
                        for (int e = PARTS - 1; e >= 0; --e) p[j] = X::mfma(v[j][m][e], b, p[j]);
                }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(s[i][g], p[j][r], acc[i][j][r]);
            }
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
    // the join: partial sums of every wavefront, added in their order, by rows, four
    // columns a thread
    constexpr int TILES = NT * MT, JR = S::JOIN_ROW;
    float* part = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                part[((wave * TILES + i * MT + j) * 16 + 4 * fq + r) * JR + fr] = acc[i][j][r];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < (TILES + W - 1) / W; ++u) {
        const int at = u * (64 * W) + (int)threadIdx.x, row = at / (4 * NT), four = at % (4 * NT);
        const int64_t n = n0 + 4 * four;
        if (row >= rows || n >= N) continue;
        const float* p = part + (((four >> 2) * MT + (row >> 4)) * 16 + (row & 15)) * JR + 4 * (four & 3);
        f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 o = *reinterpret_cast<const f32x4*>(p + w * (TILES * 16 * JR));
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += o[r];
        }
        store(row, n, v, N - n < 4 ? (int)(N - n) : 4);
    }
}

}  // namespace gqg4
