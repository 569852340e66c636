// gq_g4_dx.hip -- gradient of the products with 4-bit weights with respect to X
// (gfx950), of one matrix or of an expert each.
//
// dX[m][k] = sum_n s[n][k / G] (q[n][k] - z[n][k / G]) dY[m][n]: the scales vary
// along the sum, so each weight is formed first, exactly, and rounded to 16 bits
// for the matrix cores.  W^T is the A operand and dY the B operand, so that a lane
// holds 16 neighbouring columns of one row of dX.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_f8_stream.h"
#include "gq_g4_device.h"
#include "gq_g4_dx_stream.h"
#include "gq_g4_internal.h"
#include "gq_g4_tile.h"

using namespace gqg4;

namespace {

constexpr int BK = 64;     // rows of W (columns of dY) of a stage
constexpr int STAGES = 3;  // in LDS

struct Rows {
    const uint16_t* dY;
    int64_t M, lddy;
    uint16_t* dX;
    int64_t lddx;
    int n_experts;
    const int32_t* offsets;
};

// Bound by forming the weights and by the wait at each stage, matrix cores busy 34% of
// the time: 24,120 rows of 128 experts, 704 x 2816, in 145 to 152 us (640 TFLOP/s), 3015 x
// 17408 x 5120 in 522 to 539 us (1.0 PFLOP/s, where there are 272 stages).  32 x 32 instructions,
// which gained a sixth in the product, would leave a lane two columns instead of four,
// with twice the reads of LDS.
//
// BM = 16 MT rows by BN columns, 64 a wavefront; KS = 2: two wavefronts have the
// same columns and half of the sum each.  DMA: rows of dY are whole 16-byte pieces,
// copied straight to LDS; otherwise they go through registers, element by element at
// their end.
template <typename T, int MT, int KS, bool DMA>
struct Tile {
    static constexpr int BM = 16 * MT, BN = 256 / KS;
    static constexpr int XB = BM * 128, WB = BK * (BN / 2), STAGE = XB + WB;
    static constexpr int XI = BM / 32, WI = 2 / KS;
    // scales of a wavefront's 64 columns (two groups at most) and a stage's 64 rows, two stages
    static constexpr int SCALES = 2 * 2 * BK * 8;
    static constexpr int BYTES = STAGES * STAGE + 4 * SCALES;
    static_assert(KS == 1 || 2 * 4096 * MT <= BYTES, "the join");

    static __device__ __forceinline__ void run(const G4Weights& wt, const uint16_t* __restrict__ dy, int64_t lddy,
                                               int rows, uint16_t* __restrict__ dx, int64_t lddx, int64_t k0,
                                               uint8_t* smem) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wn = wave % (4 / KS), ks = wave / (4 / KS);
        const int fr = lane & 15, fq = lane >> 4;
        const int64_t N = wt.N, K = wt.K, row_bytes = K / 2, KG = (K + wt.group - 1) / wt.group;
        const int S = (int)((N + BK - 1) / BK);

        // dY: rows of 128 bytes, chunks swizzled by row pairs; wavefront w has rows 8 (w + 4
        // u) .. + 7, from a resource of their own (zeros past the last row and past N)
        const int xr8 = lane >> 3, xlr = 8 * wave + xr8, xchunk = 8 * ((lane & 7) ^ ((xlr >> 1) & 7));  // (elements)
        // W.  The four rows, 8 apart, that the lanes read at once have to be in different
        // banks.  KS = 1: rows of 128 bytes, whose 32-byte pieces are exchanged by r / 8;
        // KS = 2: rows of 64 bytes, row 32 h + 8 a + b of the stage at 32 h + 4 b + a.
        u32x4 held[DMA ? 1 : XI];  // rows on their way through registers
        auto load = [&](int s) __attribute__((always_inline)) {
            uint8_t* d = smem + (s % STAGES) * STAGE;
            const int64_t n = (int64_t)s * BK;
            const int left = n < N ? (int)(N - n < BK ? N - n : BK) : 0;
#pragma unroll
            for (int u = 0; u < XI; ++u) {
                uint8_t* l = d + (wave + 4 * u) * 1024;
                const int first = 8 * wave + 32 * u, have = rows - first < 8 ? rows - first : 8;
                if constexpr (DMA) {
                    const Rsrc xr = make_rsrc(dy + (have > 0 ? first * lddy : 0),
                                              have > 0 ? ((have - 1) * lddy + N) * 2 : 0);
                    copy16(xr, within((uint32_t)(xr8 * lddy + xchunk) * 2, xchunk, left), l, (uint32_t)(2 * n));
                } else {
                    const uint16_t* p = dy + (first + xr8 < rows ? first + xr8 : rows - 1) * lddy + n + xchunk;
                    u32x4 v{};
                    if (xchunk + 8 <= left) {
                        __builtin_memcpy(&v, p, 16);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (xchunk + i < left) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
                    }
                    held[u] = v;
                }
            }
            const Rsrc wr = make_rsrc(wt.W + n * row_bytes + k0 / 2, left ? left * row_bytes - k0 / 2 : 0);
#pragma unroll
            for (int u = 0; u < WI; ++u) {
                int r, chunk;
                if constexpr (KS == 1) {
                    r = 8 * (wave + 4 * u) + (lane >> 3);
                    chunk = 16 * ((lane & 7) ^ (2 * ((r >> 3) & 3)));
                } else {
                    const int at = 16 * wave + (lane >> 2);
                    r = (at & 32) + 8 * (at & 3) + ((at >> 2) & 7);
                    chunk = 16 * (lane & 3);
                }
                copy16(wr, within((uint32_t)(r * row_bytes) + chunk, chunk, (int)(K - k0 < BN ? K - k0 : BN) / 2),
                       d + XB + (wave + 4 * u) * 1024);
            }
        };
        // what the last load brought (its stage's copies, WI, are younger)
        auto put_rows = [&](int s) __attribute__((always_inline)) {
            if constexpr (!DMA) {
                uint8_t* d = smem + (s % STAGES) * STAGE;
#pragma unroll
                for (int u = 0; u < XI; ++u) reinterpret_cast<u32x4*>(d + (wave + 4 * u) * 1024)[lane] = held[u];
            }
        };
        // Scales: lane l has row n + l of the stage; as T::affine gives them in LDS, [group][row].
        float* panel = reinterpret_cast<float*>(smem + STAGES * STAGE + wave * SCALES);
        const int64_t kw = k0 + 64 * wn < K ? k0 + 64 * wn : K - 1;  // (columns past K are not stored)
        const int64_t g0 = kw / wt.group, g1 = wt.group == 32 && g0 + 1 < KG ? g0 + 1 : g0;
        const uint8_t* zeros = wt.zeros ? wt.zeros : reinterpret_cast<const uint8_t*>(wt.scales);
        struct Scale {
            uint32_t s[2], z[2];
        };
        bool in = false;  // row n + lane is one of W's
        auto load_scales = [&](int s, Scale& c) __attribute__((always_inline)) {
            // (no branch: four loads each time.  Without zero points their place is read in
            // the scales, which are twice as many bytes)
            const int64_t n = (int64_t)s * BK + lane;
            in = n < N;
            const int64_t at = (in ? n : 0) * KG;
            c.s[0] = wt.scales[at + g0];
            c.s[1] = wt.scales[at + g1];
            c.z[0] = zeros[at + g0];
            c.z[1] = zeros[at + g1];
        };
        auto put_scales = [&](int s, const Scale& c) __attribute__((always_inline)) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float f = in ? scale_f32(c.s[g], wt.s_f16) : 0.0f;
                const gqf8::f32x2 v = T::affine(f, wt.zeros ? c.z[g] & 15u : 8u);
                float* p = panel + ((s & 1) * 2 + g) * (2 * BK) + 2 * lane;
                p[0] = v.x;
                p[1] = v.y;
            }
        };
        f32x4 acc[4][MT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[t][j] = f32x4{};
        const int x_half[2] = {gqf8::pos128(fr, fq), gqf8::pos128(fr, 4 + fq)};
        // lane: columns 64 wn + 4 fr .. + 3 (two bytes), rows 32 h + 8 fq .. + 7, ROW bytes apart
        constexpr int ROW = KS == 1 ? 128 : 256, HALF = 32 * (BN / 2);
        const int wat = KS == 1 ? 8 * fq * 128 + (wn ^ fq) * 32 + 2 * fr : fq * 64 + wn * 32 + 2 * fr;
        const int gsel = wt.group == 32 ? fr >> 3 : 0;
        uint32_t w[4][2];  // the bytes of rows 2 i and 2 i + 1
        f32x4 f[4];        // (T::affine) of them
        auto read_raw = [&](int s, int buf, int h, int i) __attribute__((always_inline)) {
            const uint8_t* wd = smem + buf * STAGE + XB + HALF * h + wat;
            const f32x4* sp = reinterpret_cast<const f32x4*>(panel + ((s & 1) * 2 + gsel) * (2 * BK) +
                                                             2 * (32 * h + 8 * fq));
            w[i][0] = *reinterpret_cast<const uint16_t*>(wd + 2 * ROW * i);
            w[i][1] = *reinterpret_cast<const uint16_t*>(wd + 2 * ROW * i + ROW);
            f[i] = sp[i];
        };
        auto read_x = [&](int buf, int h, int j) __attribute__((always_inline)) {
            const u32x4* d = reinterpret_cast<const u32x4*>(smem + buf * STAGE);
            return __builtin_bit_cast(typename T::x8, d[128 * j + x_half[h]]);
        };
        // rows 2 i and 2 i + 1 of the operands of the four columns
        auto expand = [&](u32x4 (&a)[4], int i) __attribute__((always_inline)) {
            weights_2x4<T>(w[i][0], w[i][1], f[i], a, i);
        };
        // A half of a stage (KS = 2: this wavefront's), whose operands a and rows b are in
        // registers: the next half's operands are formed while these are multiplied, its
        // rows read as the last products need b no more.  The barrier before a stage's last
        // products says two things: the next stage has landed for everyone, and nobody
        // needs this one's buffer, into which the one STAGES ahead is sent.
        Scale sc;
        if (S > 0) {
            load_scales(0, sc);
#pragma unroll
            for (int s = 0; s < STAGES - 1; ++s) {
                load(s);
                put_rows(s);
            }
            put_scales(0, sc);
            load_scales(1, sc);
            load(STAGES - 1);  // (the same order as in the loop, for the waits that the compiler counts)
            if constexpr (DMA) wait_copies<(STAGES - 1) * (XI + WI) + 4>();
            else wait_copies<0>();  // (the rows' loads are not counted: at an end there are others)
            gqd::lds_barrier();
            u32x4 a[4];
            typename T::x8 b[MT];
            const int h0 = KS == 1 ? 0 : ks;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                read_raw(0, 0, h0, i);
                expand(a, i);
            }
#pragma unroll
            for (int j = 0; j < MT; ++j) b[j] = read_x(0, h0, j);
            int buf = 0;
            for (int s = 0; s < S; ++s) {
                const int nbuf = buf + 1 == STAGES ? 0 : buf + 1;
#pragma unroll
                for (int hh = 0; hh < 2 / KS; ++hh) {
                    const bool last = hh == 2 / KS - 1;  // of the stage
                    if (last) {
                        // until stage s + 1 has landed: the copies of s + 2 and four loads of
                        // scales are younger
                        // (the register form: all but the copies of s + 2, so that its rows are there too)
                        if constexpr (DMA) wait_copies<(STAGES - 2) * (XI + WI) + 4>();
                        else wait_copies<WI>();
                        put_rows(s + 2);
                        put_scales(s + 1, sc);
                        load_scales(s + 2, sc);
                        gqd::lds_barrier();
                        load(s + STAGES);
                    }
                    const int nh = last ? h0 : 1, from = last ? nbuf : buf;
                    u32x4 next[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        // (one read ahead; the first products have no operand formed beside them)
                        __builtin_amdgcn_sched_barrier(0);
                        if (t == 0) read_raw(last ? s + 1 : s, from, nh, 0);
                        if (t < 3) read_raw(last ? s + 1 : s, from, nh, t + 1);
                        if (t > 0) expand(next, t - 1);
                        if (t == 3) expand(next, 3);
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            acc[t][j] = T::mfma(__builtin_bit_cast(typename T::x8, a[t]), b[j], acc[t][j]);
                            if (t == 3) b[j] = read_x(from, nh, j);
                        }
                        if (t == 3) {
                            // (formed here, not behind the next barrier)
#pragma unroll
                            for (int i = 0; i < 4; ++i) __asm__ volatile("" : "+v"(next[i]));
                        }
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // MFMA
                            if (t < 3) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);       // LDS reads
                            if (t == 3) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                            if (t > 0 && t < 3) __builtin_amdgcn_sched_group_barrier(0x002, 24 / MT, 0);  // VALU
                            if (t == 3) __builtin_amdgcn_sched_group_barrier(0x002, 48 / MT, 0);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) a[t] = next[t];
                }
                buf = nbuf;
            }
        }
        wait_copies<0>();
        if constexpr (KS == 2) {
            // the second half's sums to the wavefronts of the first
            __syncthreads();
            f32x4* part = reinterpret_cast<f32x4*>(smem) + wn * (4 * MT * 64) + lane;
            if (ks == 1) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < MT; ++j) part[64 * (t * MT + j)] = acc[t][j];
            }
            __syncthreads();
            if (ks == 1) return;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const f32x4 o = part[64 * (t * MT + j)];
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[t][j][r] += o[r];
                }
        }
        // lane: columns 64 wn + 16 fq .. + 15 of row 16 j + fr: 4 r + t
        const int64_t k = k0 + 64 * wn + 16 * fq;
        if (k >= K) return;  // (K is a multiple of 32)
        const bool vec = (lddx & 7) == 0;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row = 16 * j + fr;
            if (row >= rows) continue;
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t][j] = in_unit<T>(acc[t][j]);
            uint16_t* p = dx + (int64_t)row * lddx + k;
            if (vec) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = T::pack(acc[2 * i & 2][j][2 * h + (i >> 1)], acc[(2 * i & 2) + 1][j][2 * h + (i >> 1)]);
                    reinterpret_cast<u32x4*>(p)[h] = v;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = T::narrow(acc[i & 3][j][i >> 2]);
            }
        }
    }
};

// The launch has the tiles from number `first` on.
template <typename T, int MT, int KS, bool DMA>
__global__ __launch_bounds__(256, 2) void k_g4_dx(G4Weights wt, Rows a, int gm, int gn, int64_t first) {
    using U = Tile<T, MT, KS, DMA>;
    extern __shared__ __align__(16) uint8_t smem[];
    RowTile t{0, 0, 0};
    int tn = 0;
    if (a.offsets) {
        auto pick = [&](int total) {
            // (the grid is sized for the most tiles there can be: only the real ones are dealt out to the XCDs)
            const int64_t real = (int64_t)(total < gm ? total : gm) * gn - first;
            if (blockIdx.x >= real) return -1;
            const int64_t id = first + xcd_order(blockIdx.x, real < gridDim.x ? (int)real : (int)gridDim.x);
            tn = (int)(id % gn);
            return (int)(id / gn);
        };
        if (!tile_of(a.offsets, a.n_experts, a.M, U::BM, pick, t)) return;
    } else {
        const int64_t id = first + xcd_order(blockIdx.x, gridDim.x);
        tn = (int)(id % gn);
        t.row0 = id / gn * U::BM;
        t.rows = a.M - t.row0 < U::BM ? (int)(a.M - t.row0) : U::BM;
    }
    const G4Weights w = of_expert(wt, t.e);
    const uint16_t* dy = a.dY + t.row0 * a.lddy;
    uint16_t* dx = a.dX + t.row0 * a.lddx;
    if constexpr (MT == 8) {
        if (a.offsets && t.rows <= 64) {  // an expert's last rows
            Tile<T, 4, KS, DMA>::run(w, dy, a.lddy, t.rows, dx, a.lddx, (int64_t)tn * U::BN, smem);
            return;
        }
    }
    U::run(w, dy, a.lddy, t.rows, dx, a.lddx, (int64_t)tn * U::BN, smem);
}

// Workgroup: columns blockIdx.x % gn, row tile / gn.
template <typename T, int MT, int W, int H, int C>
__global__ __launch_bounds__(64 * W) void k_g4_dx_few(G4Weights wt, Rows a, int gm, int gn) {
    using U = DxStream<MT, W, H, C>;
    extern __shared__ __align__(16) uint8_t smem[];
    RowTile t{0, 0, 0};
    int tn = 0;
    if (a.offsets) {
        auto pick = [&](int total) {
            const int64_t real = (int64_t)(total < gm ? total : gm) * gn;
            if (blockIdx.x >= real) return -1;
            const int id = xcd_order(blockIdx.x, (int)real);
            tn = id % gn;
            return id / gn;
        };
        if (!tile_of(a.offsets, a.n_experts, a.M, U::BM, pick, t)) return;
    } else {
        const int id = xcd_order(blockIdx.x, gm * gn);
        tn = id % gn;
        t.row0 = (int64_t)(id / gn) * U::BM;
        t.rows = a.M - t.row0 < U::BM ? (int)(a.M - t.row0) : U::BM;
    }
    dx_stream<T, MT, W, H, C>(of_expert(wt, t.e), a.dY + t.row0 * a.lddy, a.lddy, t.rows, a.dX + t.row0 * a.lddx, a.lddx,
                           (int64_t)tn * U::BN, smem);
}

template <typename T, int MT, int W, int H, int C>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    using U = DxStream<MT, W, H, C>;
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, U::BM) : (a.M + U::BM - 1) / U::BM;
    const int64_t gn = (w.K + U::BN - 1) / U::BN;
    if (!grid_ok(gm * gn, 64 * W)) return hipErrorInvalidValue;  // (never: at most four times the groups below)
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_g4_dx_few<T, MT, W, H, C>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, U::BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_g4_dx_few<T, MT, W, H, C>), dim3((unsigned)(gm * gn)), dim3(64 * W), U::BYTES, s, w, a, (int)gm,
                       (int)gn);
    return hipGetLastError();
}

template <typename T, int MT, int KS, bool DMA>
hipError_t launch(const G4Weights& w, const Rows& a, hipStream_t s) {
    using U = Tile<T, MT, KS, DMA>;
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, U::BM) : (a.M + U::BM - 1) / U::BM;
    const int64_t gn = (w.K + U::BN - 1) / U::BN;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_g4_dx<T, MT, KS, DMA>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, U::BYTES);
    for (int64_t first = 0; first < gm * gn && e == hipSuccess; first += MOST_GROUPS) {
        const int64_t left = gm * gn - first;
        hipLaunchKernelGGL((k_g4_dx<T, MT, KS, DMA>), dim3((unsigned)(left < MOST_GROUPS ? left : MOST_GROUPS)),
                           dim3(256), U::BYTES, s, w, a, (int)gm, (int)gn, first);
        e = hipGetLastError();
    }
    return e;
}

// Shape of the tiles (us; rows x sum x columns).  128 x 256 where they fill half of the
// CUs (24,120 rows of 128 experts x 704 x 2816: 149, 64 rows 187; 1024 x 17408 x 5120:
// 317, 64 rows 354); otherwise more and smaller ones with the sum in two halves: 64 x
// 128 (256 x 17408 x 5120: 168, 128 x 256 314); up to 32 rows of many experts 32 x 256
// (2048 rows of 128 experts x 704 x 2816: 49, 64 x 256 56).  Rows that go through
// registers leave none for 128.
template <typename T, bool DMA>
hipError_t launch(const G4Weights& w, const Rows& a, hipStream_t s) {
    const int64_t per = a.M / a.n_experts;  // rows an expert has
    const int64_t experts = a.n_experts < a.M ? a.n_experts : a.M;
    auto tiles = [&](int64_t rows) { return (per / rows + 1) * experts * ((w.K + 255) / 256); };
    if (per <= 32) return launch<T, 2, 1, DMA>(w, a, s);
    if (tiles(128) < 128) return launch<T, 4, 2, DMA>(w, a, s);
    if constexpr (DMA) {
        if (per > 64) return launch<T, 8, 1, DMA>(w, a, s);
    }
    return launch<T, 4, 1, DMA>(w, a, s);
}

template <typename T>
hipError_t launch(const G4Weights& w, const Rows& a, hipStream_t s) {
    // Few rows (us; sum x columns): streamed by 16 wavefronts with 16 rows where there are few
    // workgroups (16 rows x 17408 x 5120: 53, four wavefronts with 32 rows 61, tiles 139; x
    // 9728 x 2560: 28, 36, 78), of 32 columns each where that leaves half of the CUs idle (44
    // and 24; one row 37 and 20, with 64 columns 47 and 24), by four with 32 rows up to two a
    // CU (32 x 2560 x 9728: 14, 16 of 16 23, tiles 24; 128 x 17408 x 5120: 111, 142, 158; 256
    // x 17408 x 5120: 182, 259, 158); experts with a row or two, up to eight a CU (96 rows of
    // 128, 2816 x 704: 26, tiles 38; 96 of 128, 704 x 2816, 4224 workgroups: 35, 22).
    const int64_t per = (a.M + a.n_experts - 1) / a.n_experts, experts = a.n_experts < a.M ? a.n_experts : a.M;
    auto groups = [&](int64_t rows) { return (per + rows - 1) / rows * experts * ((w.K + 63) / 64); };
    if (groups(16) <= 128) return few<T, 1, 16, 2, 32>(w, a, s);
    if (groups(16) <= 256) return few<T, 1, 16, 2, 64>(w, a, s);
    if (groups(32) <= (a.n_experts > 1 && per <= 2 ? 2048 : 512)) return few<T, 2, 4, 2, 64>(w, a, s);
    // (copies address eight rows in 31 bits)
    return w.N % 8 == 0 && a.lddy % 8 == 0 && a.lddy < (1 << 26) ? launch<T, true>(w, a, s) : launch<T, false>(w, a, s);
}

}  // namespace

hipError_t gqk_g4_matmul_dx(const G4Weights& w, const void* dY, int dtype, int64_t M, int64_t lddy, void* dX,
                            int64_t lddx, int n_experts, const int32_t* offsets, hipStream_t s) {
    const Rows a{static_cast<const uint16_t*>(dY), M, lddy, static_cast<uint16_t*>(dX), lddx, n_experts, offsets};
    return dtype == gqd::DT_BF16 ? launch<Bf16>(w, a, s) : launch<F16>(w, a, s);
}
