// gq_g4_matmul.hip -- product of many rows with 4-bit weights and group scales on
// the matrix cores (gfx950), of one matrix or of an expert each.
//
// Y[m][n] = sum over groups g of s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) X[m][k].
// W is the A operand of the matrix instructions and X the B operand, so that a
// lane holds neighbouring columns of one row of Y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_g4_device.h"
#include "gq_g4_internal.h"
#include "gq_g4_stream.h"
#include "gq_g4_tile.h"

using namespace gqg4;

namespace {

struct Rows {
    const void* X;
    int64_t M, ldx;
    void* Y;
    int64_t ldy;
    int y_f32, n_experts;
    const int32_t* offsets;
};

// ------------------------------------------------------------- few rows ----

template <typename X, bool ZP, int G, int NT, int W, int XR>
__global__ __launch_bounds__(64 * W) void k_g4_few(G4Weights wt, Rows a) {
    using S = StreamSize<X, NT, XR>;
    __shared__ __align__(16) uint8_t smem[W * (S::BYTES > S::JOIN ? S::BYTES : S::JOIN)];
    RowTile t{0, 0, 0};
    if (a.offsets) {
        if (!tile_of(a.offsets, a.n_experts, a.M, XR, [&](int) { return (int)blockIdx.y; }, t)) return;
    } else {
        t.row0 = (int64_t)blockIdx.y * XR;
        t.rows = a.M - t.row0 < XR ? (int)(a.M - t.row0) : XR;
    }
    const int y_dtype = a.y_f32 ? gqd::DT_F32 : X::dtype;
    stream_tile<X, ZP, G, NT, W, XR>(of_expert(wt, t.e), (int64_t)blockIdx.x * (16 * NT),
                                     static_cast<const uint16_t*>(a.X) + t.row0 * a.ldx, a.ldx, t.rows, smem,
                                     [&](int i, int64_t n, float v) {
                                         store_as(a.Y, (t.row0 + i) * a.ldy + n, y_dtype, v);
                                     });
}

// ------------------------------------------------------- many rows (tiles) ----

constexpr int BK = 64;     // inputs of a stage
constexpr int STAGES = 3;  // in LDS

// Eight weights s (q - z) of a dword, rounded to 16 bits; s512 = 512 s, sz = -z s.
// A nibble as an e4m3 byte is q 2^-9 (subnormal below 8, the first normal binade
// from 8 on), which one instruction converts two at a time; s (q - z) is exact in
// fp32 (16 bits), so the one rounding is the last.
template <typename T>
__device__ __forceinline__ typename T::x8 weights8(uint32_t w, float s512, float sz) {
    const int lo = (int)(w & 0x0f0f0f0fu), hi = (int)((w >> 4) & 0x0f0f0f0fu);
    const gqf8::f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(lo, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(lo, true);
    const gqf8::f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(hi, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(hi, true);
    auto f = [&](float q) { return __builtin_fmaf(q, s512, sz); };
    return __builtin_bit_cast(typename T::x8, u32x4{T::pack(f(a.x), f(c.x)), T::pack(f(a.y), f(c.y)),
                                                   T::pack(f(b.x), f(d.x)), T::pack(f(b.y), f(d.y))});
}

// BM = 16 MT rows of X by BN = 64 NT columns; four wavefronts, each all the rows
// by a quarter of the columns, so that a weight is expanded by one wavefront only,
// in registers, right before the matrix instructions that use it.  Both operands
// of a stage of 64 inputs go to LDS as they are in memory, STAGES ahead.
template <typename T, int MT, int NT>
struct Tile {
    static constexpr int BM = 16 * MT, BN = 64 * NT;
    static constexpr int XB = BM * 128, WB = BN * 32, STAGE = XB + WB;
    static constexpr int XI = BM / 32, WI = BN / 128, LOADS = XI + WI;  // copies of a wavefront
    static constexpr int PANEL = 4 * 16 * NT * 8;                       // scales of a wavefront
    static constexpr int BYTES = STAGES * STAGE + 4 * PANEL;
    static_assert(MT % 2 == 0 && NT % 2 == 0, "whole copies");

    // x: first row of the tile; n0: first column
    static __device__ __forceinline__ void run(const G4Weights& wt, const uint16_t* __restrict__ x, int64_t ldx,
                                               int rows, void* __restrict__ y, int64_t ldy, int y_f32, int64_t n0,
                                               uint8_t* smem) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int fr = lane & 15, fq = lane >> 4;
        const int64_t N = wt.N, K = wt.K, row_bytes = K / 2;
        const int S = (int)((K + BK - 1) / BK), KG = (int)((K + wt.group - 1) / wt.group);
        const int64_t w_rows = N - n0 < BN ? N - n0 : BN;
        const Rsrc wr = make_rsrc(wt.W + n0 * row_bytes, w_rows * row_bytes);
        const Rsrc xr = make_rsrc(x, ((rows - 1) * ldx + K) * 2);

        // X: rows of 128 bytes, chunks swizzled by row pairs; wavefront w brings rows 8 (w + 4 u) .. + 7
        uint32_t xoff[XI];
        const int xlr = 8 * wave + (lane >> 3), xchunk = 16 * ((lane & 7) ^ ((xlr >> 1) & 7));
#pragma unroll
        for (int u = 0; u < XI; ++u) {
            const int r = xlr + 32 * u;
            xoff[u] = (uint32_t)((r < rows ? r : rows - 1) * ldx * 2) + xchunk;
        }
        // W: two chunks a row, 32 rows a copy, each wavefront its own columns (so that
        // they wait for no other's).  An operand's rows are 32 p + 8 (a / 4) + 4 o + a %
        // 4 (a = l % 16, tile 2 p + o): row r sits at pair x = 16 o + 8 (a / 8) + a % 8
        // of its copy, its chunks exchanged where a >= 8, so that 16 rows at one chunk
        // cover all banks.
        const int wx = lane >> 1, wa = wx & 15;
        const int wrow = 8 * (wa >> 2) + 4 * (wx >> 4) + (wa & 3);
        const int wchunk = 16 * ((lane & 1) ^ (wa >> 3));
        uint32_t woff[WI];
#pragma unroll
        for (int u = 0; u < WI; ++u) woff[u] = (uint32_t)((32 * (WI * wave + u) + wrow) * row_bytes) + wchunk;
        int lg = 0;
        auto load = [&](int s) {
            uint8_t* d = smem + lg * STAGE;
            lg = lg + 1 == STAGES ? 0 : lg + 1;
            const int64_t k = (int64_t)s * BK;
            const int left = k < K ? (int)(K - k < BK ? K - k : BK) : 0;
#pragma unroll
            for (int u = 0; u < WI; ++u)
                copy16(wr, within(woff[u], wchunk, left / 2), d + XB + (WI * wave + u) * 1024, (uint32_t)(k / 2));
#pragma unroll
            for (int u = 0; u < XI; ++u)
                copy16(xr, within(xoff[u], xchunk, 2 * left), d + (wave + 4 * u) * 1024, (uint32_t)(2 * k));
        };

        // Scales: lane l < 16 NT loads those of the column n0 + 16 NT wave + l, four
        // groups at a time, and puts 512 s and -z s into LDS ([group][column], each
        // wavefront its own), where the lanes that use them read them.
        const int64_t sn = n0 + 16 * NT * wave + (lane < 16 * NT ? lane : 0);
        const int64_t srow = (sn < N ? sn : N - 1) * KG;
        float* panel = reinterpret_cast<float*>(smem + STAGES * STAGE + wave * PANEL);
        uint32_t four_a, four_b, four_z;
        auto load_four = [&](int g0) {
            four_a = four_b = 0;
            four_z = 0x08080808u;
            if (g0 + 4 <= KG) {
                u32x2 v;
                __builtin_memcpy(&v, wt.scales + srow + g0, 8);
                four_a = v.x;
                four_b = v.y;
                if (wt.zeros) __builtin_memcpy(&four_z, wt.zeros + srow + g0, 4);
            } else if (g0 < KG) {
                const int n = KG - g0;
                four_a = wt.scales[srow + g0];
                if (n > 1) four_a |= (uint32_t)wt.scales[srow + g0 + 1] << 16;
                if (n > 2) four_b = wt.scales[srow + g0 + 2];
                if (wt.zeros) {
                    four_z = wt.zeros[srow + g0];
                    if (n > 1) four_z |= (uint32_t)wt.zeros[srow + g0 + 1] << 8;
                    if (n > 2) four_z |= (uint32_t)wt.zeros[srow + g0 + 2] << 16;
                }
            }
        };
        auto put_four = [&]() {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float f = scale_f32(((g & 2 ? four_b : four_a) >> (16 * (g & 1))) & 0xffffu, wt.s_f16);
                gqf8::f32x2 v;
                v.x = 512.0f * f;
                v.y = -(float)((four_z >> (8 * g)) & 15u) * f;
                if (lane < 16 * NT) reinterpret_cast<gqf8::f32x2*>(panel)[16 * NT * g + lane] = v;
            }
        };
        const int gshift = wt.group == 32 ? 0 : wt.group == 64 ? 1 : 2;  // half stages of a group
        const int per4 = 2 << gshift;                                    // stages of four groups

        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{};
        // Operand c of a stage: the 32 inputs of its half c / NT, tile c % NT.  A lane
        // has the eight of dword fq of the half's chunk; of X the chunk 4 (c / NT) + fq.
        const int wbase = XB + 16 * NT * wave * 32 + 32 * fr + 4 * fq;
        const int w_half[2] = {wbase + 16 * (fr >> 3), wbase + 16 * (1 - (fr >> 3))};
        const int x_half[2] = {gqf8::pos128(fr, fq), gqf8::pos128(fr, 4 + fq)};
        const gqf8::f32x2* pbase = reinterpret_cast<const gqf8::f32x2*>(panel) + 8 * (fr >> 2) + (fr & 3);
        struct Raw {
            uint32_t w;
            gqf8::f32x2 s;
        };
        auto read_raw = [&](int buf, int s, int c, Raw& r) {
            const int i = c % NT, h = c / NT;
            r.w = *reinterpret_cast<const uint32_t*>(smem + buf * STAGE + w_half[h] + 1024 * (i >> 1) + 512 * (i & 1));
            r.s = pbase[16 * NT * (((2 * s + h) >> gshift) & 3) + 32 * (i >> 1) + 4 * (i & 1)];
        };
        auto read_x = [&](int buf, int h, typename T::x8 (&b)[MT]) {
            const u32x4* d = reinterpret_cast<const u32x4*>(smem + buf * STAGE);
#pragma unroll
            for (int j = 0; j < MT; ++j) b[j] = __builtin_bit_cast(typename T::x8, d[128 * j + x_half[h]]);
        };
        // A stage, whose rows b0 of the first half, first operand a and second one's
        // bytes are in registers: each operand is formed while the one before it is
        // multiplied, its bytes read while the one before that is.  The barrier before
        // the last products says two things: the next stage's rows have landed for
        // everyone, and nobody needs this stage's buffer, into which the one STAGES
        // ahead is sent.
        if (S > 0) {
            load_four(0);
#pragma unroll
            for (int s = 0; s < STAGES; ++s) load(s);
            put_four();
            load_four(4);
            wait_copies<(STAGES - 1) * LOADS>();
            gqd::lds_barrier();
            typename T::x8 b0[MT], b1[MT], a;
            Raw r[2];
            read_raw(0, 0, 0, r[0]);
            read_raw(0, 0, 1, r[1]);
            read_x(0, 0, b0);
            a = weights8<T>(r[0].w, r[0].s.x, r[0].s.y);
            int buf = 0;
            for (int s = 0; s < S; ++s) {
                const int nbuf = buf + 1 == STAGES ? 0 : buf + 1;
                read_x(buf, 1, b1);
#pragma unroll
                for (int c = 0; c < 2 * NT; ++c) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (c == 2 * NT - 2) {
                        wait_copies<(STAGES - 2) * LOADS>();
                        if ((s + 1) % per4 == 0) {
                            put_four();
                            load_four(((s + 1) / per4 + 1) * 4);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (c == 2 * NT - 1) {
                        gqd::lds_barrier();
                        __builtin_amdgcn_sched_barrier(0);
                        read_x(nbuf, 0, b0);
                        load(s + STAGES);
                    }
                    // (r[(c + 1) % 2] is operand c + 1's)
                    const Raw& n = r[(c + 1) & 1];
                    const typename T::x8 next = weights8<T>(n.w, n.s.x, n.s.y);
                    if (c + 2 < 2 * NT) read_raw(buf, s, c + 2, r[c & 1]);
                    else read_raw(nbuf, s + 1, c + 2 - 2 * NT, r[c & 1]);
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[c % NT][j] = T::mfma(a, c < NT ? b0[j] : b1[j], acc[c % NT][j]);
                    a = next;
                    if (c == 2 * NT - 3) __asm__ volatile("" : "+v"(a));  // (formed here, not behind the next branch)
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        if (c == 2 * NT - 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                      // MFMA
                        if (j < 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);           // LDS reads
                        __builtin_amdgcn_sched_group_barrier(0x002, 24 / MT, 0);                // VALU
                        if (c == 2 * NT - 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0); // copies
                    }
                }
                buf = nbuf;
            }
        }
        wait_copies<0>();
        // lane: columns 32 p + 8 fq .. + 7 (tiles 2 p, 2 p + 1) of row 16 j + fr
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row = 16 * j + fr;
            if (row >= rows) continue;
#pragma unroll
            for (int i = 0; i < NT; i += 2) {
                const int64_t n = n0 + 16 * NT * wave + 16 * i + 8 * fq;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (n + r < N) {
                        const float v = r < 4 ? acc[i][j][r & 3] : acc[i + 1][j][r & 3];
                        if (y_f32) static_cast<float*>(y)[row * ldy + n + r] = v;
                        else static_cast<uint16_t*>(y)[row * ldy + n + r] = T::narrow(v);
                    }
            }
        }
    }
};

template <typename T, int MT, int NT>
__global__ __launch_bounds__(256, 2) void k_g4_tile(G4Weights wt, Rows a, int gm, int gn) {
    using U = Tile<T, MT, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    RowTile t{0, 0, 0};
    int tn = 0;
    if (a.offsets) {
        auto pick = [&](int total) {
            // (the grid is sized for the most tiles there can be: only the real ones are dealt out to the XCDs)
            const int64_t real = (int64_t)(total < gm ? total : gm) * gn;
            if (blockIdx.x >= real) return -1;
            const int id = xcd_order(blockIdx.x, (int)real);
            tn = id % gn;
            return id / gn;
        };
        if (!tile_of(a.offsets, a.n_experts, a.M, U::BM, pick, t)) return;
    } else {
        const int id = xcd_order(blockIdx.x, gm * gn);
        constexpr int BAND = 8;
        const int bands = (gm + BAND - 1) / BAND, h = (gm + bands - 1) / bands;
        const int band = id / (h * gn), hb = gm - band * h < h ? gm - band * h : h;
        const int c = id - band * h * gn;
        tn = c / hb;
        t.row0 = (int64_t)(band * h + c % hb) * U::BM;
        t.rows = a.M - t.row0 < U::BM ? (int)(a.M - t.row0) : U::BM;
    }
    U::run(of_expert(wt, t.e), static_cast<const uint16_t*>(a.X) + t.row0 * a.ldx, a.ldx, t.rows,
           a.y_f32 ? static_cast<void*>(static_cast<float*>(a.Y) + t.row0 * a.ldy)
                   : static_cast<void*>(static_cast<uint16_t*>(a.Y) + t.row0 * a.ldy),
           a.ldy, a.y_f32, (int64_t)tn * U::BN, smem);
}

template <typename T, int MT, int NT>
hipError_t tile(const G4Weights& w, const Rows& a, hipStream_t s) {
    using U = Tile<T, MT, NT>;
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, U::BM) : (a.M + U::BM - 1) / U::BM;
    const int64_t gn = (w.N + U::BN - 1) / U::BN;
    if (!grid_ok(gm * gn, 256)) return hipErrorInvalidValue;
    const int lds = U::BYTES;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_g4_tile<T, MT, NT>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_g4_tile<T, MT, NT>), dim3((unsigned)(gm * gn)), dim3(256), lds, s, w, a, (int)gm, (int)gn);
    return hipGetLastError();
}

template <typename X, bool ZP, int G, int NT, int W, int XR>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, XR) : (a.M + XR - 1) / XR;
    const int64_t gn = (w.N + 16 * NT - 1) / (16 * NT);
    if (!grid_ok(gn, 64 * W) || gm > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_g4_few<X, ZP, G, NT, W, XR>), dim3((unsigned)gn, (unsigned)gm), dim3(64 * W), 0, s, w, a);
    return hipGetLastError();
}

template <typename X, bool ZP, int G>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    return few<X, ZP, G, 2, 4, 16>(w, a, s);
}

template <typename X, bool ZP>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    if (w.group == 32) return few<X, ZP, 32>(w, a, s);
    if (w.group == 64) return few<X, ZP, 64>(w, a, s);
    return few<X, ZP, 128>(w, a, s);
}

template <typename X, typename T>
hipError_t matmul(const G4Weights& w, const Rows& a, hipStream_t s) {
    const int64_t per = a.M / a.n_experts;  // rows an expert has
    if (per <= 16 || a.y_f32) return w.zeros ? few<X, true>(w, a, s) : few<X, false>(w, a, s);
    if (per <= 64) return tile<T, 4, 4>(w, a, s);
    return tile<T, 8, 4>(w, a, s);
}

}  // namespace

hipError_t gqk_g4_matmul(const G4Weights& w, const void* X, int x_dtype, int64_t M, int64_t ldx, void* Y, int y_dtype,
                         int64_t ldy, int n_experts, const int32_t* offsets, hipStream_t s) {
    const Rows a{X, M, ldx, Y, ldy, y_dtype == gqd::DT_F32, n_experts, offsets};
    return x_dtype == gqd::DT_BF16 ? matmul<XBf16, Bf16>(w, a, s) : matmul<XF16, F16>(w, a, s);
}
