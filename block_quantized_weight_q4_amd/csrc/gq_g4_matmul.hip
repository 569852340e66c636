// gq_g4_matmul.hip -- product of many rows with 4-bit weights and group scales on
// the matrix cores (gfx950), of one matrix or of an expert each.
//
// Y[m][n] = sum over groups g of s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) X[m][k].
// W is the A operand of the matrix instructions and X the B operand, so that a
// lane holds neighbouring columns of one row of Y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// Workgroup first + blockIdx.x: columns % gn, row tile / gn.
template <typename X, bool ZP, int G, int NT, int W, int XR>
__global__ __launch_bounds__(64 * W) void k_g4_few(G4Weights wt, Rows a, int gn, int64_t first) {
    using S = StreamSize<X, NT, XR>;
    __shared__ __align__(16) uint8_t smem[W * (S::BYTES > S::JOIN ? S::BYTES : S::JOIN)];
    const int64_t id = first + blockIdx.x, tm = id / gn;
    RowTile t{0, 0, 0};
    if (a.offsets) {
        if (!tile_of(a.offsets, a.n_experts, a.M, XR, [&](int) { return (int)tm; }, t)) return;
    } else {
        t.row0 = tm * XR;
        t.rows = a.M - t.row0 < XR ? (int)(a.M - t.row0) : XR;
    }
    const int y_dtype = a.y_f32 ? gqd::DT_F32 : X::dtype;
    stream_tile<X, ZP, G, NT, W, XR>(of_expert(wt, t.e), (id - tm * gn) * (16 * NT),
                                     static_cast<const uint16_t*>(a.X) + t.row0 * a.ldx, a.ldx, t.rows, smem,
                                     [&](int i, int64_t n, f32x4 v, int c) {
                                         store_as(a.Y, (t.row0 + i) * a.ldy + n, y_dtype, v, c);
                                     });
}

// ------------------------------------------------------- many rows (tiles) ----

constexpr int BK = 64;   // inputs of a stage
constexpr int BAND = 4;  // row tiles of a band

// Eight weights of a dword, rounded to 16 bits, in T's unit; s and sz as T::affine gives them.
template <typename T>
__device__ __forceinline__ typename T::x8 weights8(uint32_t w, float s, float sz) {
    const int lo = (int)(w & 0x0f0f0f0fu), hi = (int)((w >> 4) & 0x0f0f0f0fu);
    const gqf8::f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(lo, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(lo, true);
    const gqf8::f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(hi, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(hi, true);
    auto f = [&](float q) { return __builtin_fmaf(q, s, sz); };
    return __builtin_bit_cast(typename T::x8, u32x4{T::pack(f(a.x), f(c.x)), T::pack(f(a.y), f(c.y)),
                                                   T::pack(f(b.x), f(d.x)), T::pack(f(b.y), f(d.y))});
}

// BM = 32 MT rows of X by BN = 128 NT columns; four wavefronts, each all the rows
// by a quarter of the columns, so that a weight is expanded by one wavefront only,
// in registers, right before the matrix instructions that use it.  Both operands go
// to LDS as they are in memory: X in stages of 64 inputs, W in blocks of two stages
// (64 bytes a row).
//
// Bound by the matrix cores and what they are fed with: 3015 x 17408 x 5120 takes 449 to
// 484 us (1.11 to 1.20 PFLOP/s; a library's product of the same rows with expanded
// weights 505, of 8192^3 1.13 to 1.33 PFLOP/s, depending on the card and its heat), with
// the matrix cores busy 72% of the time and 60% of the issue cycles spent on expanding
// (20 instructions for eight weights).  Two workgroups a CU hide each other's starts and
// ends; eight wavefronts in one, 16 x 16 instructions (576 us) and two barriers a stage
// (703 us) were slower.  Short sums are bound by those starts and by the stores: 24,120
// rows of 128 experts, 2816 x 704 (11 stages a tile), 136 to 147 us, 650 to 700 TFLOP/s.
template <typename T, int MT, int NT>
struct Tile {
    static constexpr int NW = 4, XS = 2;  // wavefronts, stages of X
    static constexpr int BM = 32 * MT, BN = 32 * NT * NW;
    static constexpr int XB = BM * 128, WB = BN * 64;
    static constexpr int XI = BM / 8 / NW, WI = 2 * NT;  // copies of a wavefront
    static constexpr int PANEL = 32 * NT * 8;         // scales of a wavefront
    static constexpr int W_AT = XS * XB, P_AT = W_AT + 2 * WB, BYTES = P_AT + NW * PANEL;
    static_assert(BM % (8 * NW) == 0 && NT <= 2, "whole copies, a lane a column");

    // x: first row of the tile; n0: first column
    static __device__ __forceinline__ void run(const G4Weights& wt, const uint16_t* __restrict__ x, int64_t ldx,
                                               int rows, uint16_t* __restrict__ y, int64_t ldy, int64_t n0,
                                               uint8_t* smem) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int fr = lane & 31, fq = lane >> 5;
        const int64_t N = wt.N, K = wt.K, row_bytes = K / 2;
        const int S = (int)((K + BK - 1) / BK), KG = (int)((K + wt.group - 1) / wt.group);
        const int64_t w_rows = N - n0 < BN ? N - n0 : BN;
        const Rsrc wr = make_rsrc(wt.W + n0 * row_bytes, w_rows * row_bytes);
        const Rsrc xr = make_rsrc(x, ((rows - 1) * ldx + K) * 2);

        // X: rows of 128 bytes, chunks swizzled by row pairs; wavefront w brings rows 8 (w + NW u) .. + 7
        uint32_t xoff[XI];
        const int xlr = 8 * wave + (lane >> 3), xchunk = 16 * ((lane & 7) ^ ((xlr >> 1) & 7));
#pragma unroll
        for (int u = 0; u < XI; ++u) {
            const int r = xlr + 8 * NW * u;
            xoff[u] = (uint32_t)((r < rows ? r : rows - 1) * ldx * 2) + xchunk;
        }
        // W: each wavefront its own columns (so that they wait for no other's), 16 rows of
        // four chunks a copy, chunk c of row r at c ^ (r / 4), so that 16 rows at one chunk
        // cover all banks
        const int cr = lane >> 2, wchunk = 16 * ((lane & 3) ^ (cr >> 2));
        uint32_t woff[WI];
#pragma unroll
        for (int u = 0; u < WI; ++u) woff[u] = (uint32_t)((32 * NT * wave + 16 * u + cr) * row_bytes) + wchunk;
        auto load_x = [&](int s, int buf) __attribute__((always_inline)) {
            const int64_t k = (int64_t)s * BK;
            const int left = k < K ? (int)(K - k < BK ? K - k : BK) : 0;
            uint8_t* d = smem + buf * XB;
#pragma unroll
            for (int u = 0; u < XI; ++u)
                copy16(xr, within(xoff[u], xchunk, 2 * left), d + (wave + NW * u) * 1024, (uint32_t)(2 * k));
        };
        auto load_w = [&](int b, int buf) __attribute__((always_inline)) {
            const int64_t k = (int64_t)b * (2 * BK);
            const int left = k < K ? (int)(K - k < 2 * BK ? K - k : 2 * BK) : 0;
            uint8_t* d = smem + W_AT + buf * WB;
#pragma unroll
            for (int u = 0; u < WI; ++u)
                copy16(wr, within(woff[u], wchunk, left / 2), d + (WI * wave + u) * 1024, (uint32_t)(k / 2));
        };

        // Scales: lane l < 32 NT has those of the column n0 + 32 NT wave + l, four groups
        // at a time, and puts T::affine of the group in use into LDS (each wavefront
        // its own), where the lanes of the operand's rows read them.
        const int64_t sn = n0 + 32 * NT * wave + (lane < 32 * NT ? lane : 0);
        const int64_t srow = (sn < N ? sn : N - 1) * KG;
        gqf8::f32x2* panel = reinterpret_cast<gqf8::f32x2*>(smem + P_AT + wave * PANEL);
        uint32_t four_a, four_b, four_z;  // groups 4 i .. 4 i + 3, the next of them lowest
        auto load_four = [&](int g0) __attribute__((always_inline)) {
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
        // group g into LDS: behind the reads of the one before it (a wavefront's LDS operations keep their order)
        auto put_scales = [&](int g) __attribute__((always_inline)) {
            const gqf8::f32x2 v = T::affine(scale_f32(four_a & 0xffffu, wt.s_f16), four_z & 15u);
            if (lane < 32 * NT) panel[lane] = v;
            four_a = (four_a >> 16) | (four_b << 16);
            four_b >>= 16;
            four_z >>= 8;
            if ((g & 3) == 3) load_four(g + 1);
        };
        const int gshift = wt.group == 32 ? 0 : wt.group == 64 ? 1 : 2;  // half stages of a group

        f32x16 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x16{};
        // Operand c of a stage: the 16 inputs of its step t = c / NT (eight of them a lane: dword
        // 2 fq + t % 2 of W's chunk t / 2, so that one read brings those of two steps, and
        // chunk 4 (t / 2) + 2 fq + t % 2 of X), tile c % NT.
        // Row a = l % 32 of a tile of W is its column 16 (a / 4 % 2) + 4 (a / 8) + a % 4, so
        // that a lane ends up with 16 neighbouring columns of one row of Y.
        const int wcol = 16 * ((fr >> 2) & 1) + 4 * (fr >> 3) + (fr & 3), wr16 = wcol & 15;
        const int wbase = W_AT + 1024 * (WI * wave + (wcol >> 4)) + 64 * wr16 + 8 * fq;
        int w_half[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) w_half[h] = wbase + 16 * (h ^ (wr16 >> 2));
        int x_step[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) x_step[t] = gqf8::pos128(fr, 4 * (t >> 1) + 2 * fq + (t & 1));
        const gqf8::f32x2* pbase = panel + wcol;
        struct Raw {
            u32x2 w;  // of two steps
            gqf8::f32x2 s;
        };
        // (h: chunk of W's block, 32 inputs: of one group)
        auto read_raw = [&](int buf, int h, int i, Raw& r) __attribute__((always_inline)) {
            r.w = *reinterpret_cast<const u32x2*>(smem + buf * WB + w_half[h] + 2048 * i);
            r.s = pbase[32 * i];
        };
        auto read_x = [&](int buf, int t, int j) __attribute__((always_inline)) {
            const u32x4* d = reinterpret_cast<const u32x4*>(smem + buf * XB);
            return __builtin_bit_cast(typename T::x8, d[256 * j + x_step[t]]);
        };
        // A stage, whose first step's rows b, first operand a and second one's bytes
        // are in registers: each operand is formed while the one before it is
        // multiplied, its bytes read while the one before that is; a step's rows are
        // read into the registers of the last step's as its last products need them no
        // more.  The barrier before a stage's last products says two things: the next
        // stage's rows have landed for everyone, and nobody needs this stage's buffer,
        // into which the one XS ahead is sent.
        if (S > 0) {
            load_four(0);
            load_w(0, 0);
#pragma unroll
            for (int s = 0; s < XS; ++s) load_x(s, s);
            load_w(1, 1);
            put_scales(0);
            wait_copies<(XS - 1) * XI + WI>();
            gqd::lds_barrier();
            typename T::x8 b[MT], a;
            Raw r[2];
            read_raw(0, 0, 0, r[0]);
            if constexpr (NT == 2) read_raw(0, 0, 1, r[1]);
#pragma unroll
            for (int j = 0; j < MT; ++j) b[j] = read_x(0, 0, j);
            a = weights8<T>(r[0].w.x, r[0].s.x, r[0].s.y);
            int buf = 0, wb = 0;  // of this stage
            auto stage = [&](int s, auto odd) __attribute__((always_inline)) {
                constexpr int C = 4 * NT;
                const int nbuf = buf + 1 == XS ? 0 : buf + 1;
                const int nwb = odd ? wb ^ 1 : wb;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    __builtin_amdgcn_sched_barrier(0);
                    // the group of the half that is read next
                    if (c == C / 2 - 2 && wt.group == 32) put_scales(2 * s + 1);
                    if (c == C - 2) {
                        // until stage s + 1 has landed
                        wait_copies<(XS - 2) * XI + (odd ? 0 : WI)>();
                        if ((2 * s + 2) % (1 << gshift) == 0) put_scales((2 * s + 2) >> gshift);
                    }
                    if (c == C - 1) {
                        gqd::lds_barrier();
                        __builtin_amdgcn_sched_barrier(0);
                        load_x(s + XS, buf);
                        if constexpr (odd) load_w((s + 3) / 2, wb);
                    }
                    // r[which(c)] has the bytes of operand c: of the two tiles in turn, with one tile of
                    // the chunks in turn.  Two operands ahead the next chunk's are read, when the others
                    // that lay there are formed.
                    auto which = [](int c) { return NT == 2 ? c & 1 : (c >> 1) & 1; };
                    const Raw& n = r[which(c + 1)];
                    const typename T::x8 next = weights8<T>((c + 1) / NT & 1 ? n.w.y : n.w.x, n.s.x, n.s.y);
                    const bool fresh = NT == 2 ? c & 2 : !(c & 1), more = c + 2 < C;  // (of this stage)
                    if (fresh) read_raw(more ? wb : nwb, more ? (odd ? 3 : 1) : (odd ? 0 : 2), c & (NT - 1), r[which(c + 2)]);
                    const bool last = c % NT == NT - 1;  // of its step
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        acc[c % NT][j] = T::mfma32(a, b[j], acc[c % NT][j]);
                        if (last) b[j] = c + 1 < C ? read_x(buf, (c + 1) / NT, j) : read_x(nbuf, 0, j);
                    }
                    a = next;
                    // (formed here, not behind the next branch)
                    if (c == C - 3 || c == C / 2 - 3) __asm__ volatile("" : "+v"(a));
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                // MFMA
                        if (fresh) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS reads
                        if (last) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);                // VALU
                        if (c == C - 1) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);  // copies
                    }
                }
                buf = nbuf;
                wb = nwb;
            };
            int s = 0;
            for (; s + 1 < S; s += 2) {
                stage(s, std::false_type{});
                stage(s + 1, std::true_type{});
            }
            if (s < S) stage(s, std::false_type{});
        }
        wait_copies<0>();
        // lane: columns 16 fq .. + 15 of the tiles of row 32 j + fr
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row = 32 * j + fr;
            if (row >= rows) continue;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int64_t n = n0 + 32 * NT * wave + 32 * i + 16 * fq;
                const f32x16 v = in_unit<T>(acc[i][j]);
                uint16_t* p = y + row * ldy + n;
#pragma unroll
                for (int r = 0; r < 16; r += 8) {
                    if (n + r + 8 <= N) {
                        const u32x4 o{T::pack(v[r], v[r + 1]), T::pack(v[r + 2], v[r + 3]),
                                      T::pack(v[r + 4], v[r + 5]), T::pack(v[r + 6], v[r + 7])};
                        __builtin_memcpy(p + r, &o, 16);  // (of any alignment)
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + r + e < N) p[r + e] = T::narrow(v[r + e]);
                    }
                }
            }
        }
    }
};

// The launch has n_full tiles from number `first` on, and workgroups from n_full on take
// halves of the tiles behind them, PARTS = 2 a tile, by columns (dense; by rows weights
// would be expanded twice): the last, partial round of tiles would take as long as a
// whole one on a part of the CUs.
template <typename T, int MT, int NT, int PARTS>
__global__ __launch_bounds__(256, 2) void k_g4_tile(G4Weights wt, Rows a, int gm, int gn, int n_full, int64_t first) {
    using U = Tile<T, MT, NT>;
    using P = Tile<T, MT, NT / PARTS>;
    extern __shared__ __align__(16) uint8_t smem[];
    RowTile t{0, 0, 0};
    int64_t n0 = 0;
    bool part = false;
    if (a.offsets) {
        auto pick = [&](int total) {
            // (the grid is sized for the most tiles there can be: only the real ones are dealt out to the XCDs)
            const int64_t real = (int64_t)(total < gm ? total : gm) * gn - first;
            if (blockIdx.x >= real) return -1;
            const int64_t id = first + xcd_order(blockIdx.x, real < n_full ? (int)real : n_full);
            n0 = id % gn * U::BN;
            return (int)(id / gn);
        };
        if (!tile_of(a.offsets, a.n_experts, a.M, U::BM, pick, t)) return;
    } else {
        int here, q = 0;
        part = PARTS > 1 && (int)blockIdx.x >= n_full;
        if (part) {
            q = ((int)blockIdx.x - n_full) % PARTS;
            here = n_full + ((int)blockIdx.x - n_full) / PARTS;
        } else {
            here = xcd_order(blockIdx.x, n_full);
        }
        const int64_t id = first + here;
        // bands of at most BAND row tiles, each walked column of tiles by column
        const int bands = (gm + BAND - 1) / BAND, h = (gm + bands - 1) / bands;
        const int band = (int)(id / (h * gn)), hb = gm - band * h < h ? gm - band * h : h;
        const int c = (int)(id % (h * gn));
        n0 = (int64_t)(c / hb) * U::BN + q * P::BN;
        if (n0 >= wt.N) return;
        t.row0 = (int64_t)(band * h + c % hb) * U::BM;
        t.rows = a.M - t.row0 < U::BM ? (int)(a.M - t.row0) : U::BM;
    }
    const G4Weights w = of_expert(wt, t.e);
    const uint16_t* x = static_cast<const uint16_t*>(a.X) + t.row0 * a.ldx;
    uint16_t* y = static_cast<uint16_t*>(a.Y) + t.row0 * a.ldy;
    if constexpr (PARTS > 1) {
        if (part) {
            P::run(w, x, a.ldx, t.rows, y, a.ldy, n0, smem);
            return;
        }
        // an expert's last rows
        if (a.offsets && t.rows <= 64) {
            Tile<T, 2, NT>::run(w, x, a.ldx, t.rows, y, a.ldy, n0, smem);
            return;
        }
        if (a.offsets && t.rows <= 96) {
            Tile<T, 3, NT>::run(w, x, a.ldx, t.rows, y, a.ldy, n0, smem);
            return;
        }
    }
    U::run(w, x, a.ldx, t.rows, y, a.ldy, n0, smem);
}

template <typename T, int MT, int NT, int PARTS>
hipError_t tile(const G4Weights& w, const Rows& a, hipStream_t s) {
    using U = Tile<T, MT, NT>;
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, U::BM) : (a.M + U::BM - 1) / U::BM;
    const int64_t gn = (w.N + U::BN - 1) / U::BN, tiles = gm * gn;
    const int64_t slots = 2 * gqk_cu_count(), tail = tiles % slots;
    const int64_t n_full = PARTS > 1 && !a.offsets && PARTS * tail <= slots ? tiles - tail : tiles;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_g4_tile<T, MT, NT, PARTS>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, U::BYTES);
    if (e != hipSuccess) return e;
    int64_t first = 0;
    do {
        const int64_t here = n_full - first < MOST_GROUPS ? n_full - first : MOST_GROUPS;
        const int64_t grid = here + (first + here == n_full ? PARTS * (tiles - n_full) : 0);
        hipLaunchKernelGGL((k_g4_tile<T, MT, NT, PARTS>), dim3((unsigned)grid), dim3(256), U::BYTES, s, w, a, (int)gm,
                           (int)gn, (int)here, first);
        e = hipGetLastError();
        first += here;
    } while (e == hipSuccess && first < n_full);
    return e;
}

template <typename X, bool ZP, int G, int NT, int W, int XR>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, XR) : (a.M + XR - 1) / XR;
    const int64_t gn = (w.N + 16 * NT - 1) / (16 * NT);
    for (int64_t first = 0; first < gm * gn; first += MOST_GROUPS) {
        const int64_t left = gm * gn - first;
        hipLaunchKernelGGL((k_g4_few<X, ZP, G, NT, W, XR>), dim3((unsigned)(left < MOST_GROUPS ? left : MOST_GROUPS)),
                           dim3(64 * W), 0, s, w, a, (int)gn, first);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Shape of the streamed tiles (us; N x K; n rows of W by m of X by w wavefronts).
// Experts with up to two rows: 32 by 4 by 2 (64 rows of 128 experts, 704 x 2816: 15.1,
// 32 by 4 by 4 15.8, 16 by 4 by 4 16.3, 32 by 16 by 2 16.4), with more 32 by 16 by 2
// (1024 rows, 704 x 2816: 41.7, with 4 wavefronts 45.9, 32 by 32 by 4 60.6).  One
// matrix: up to 16 rows 32 by 16 by 4 (17408 x 5120: 20.7, 32 by 32 by 4 25.9), of up
// to 4096 columns 16 by 16 by 4 (2560 x 9728: 9.3 and 12.5); more rows 32 by 32 by 4,
// which reads W half as often (1024 rows of 17408 x 5120: 425, 32 by 16 by 4 540).
// Where there are thousands of workgroups, nothing is left to split: one wavefront a
// workgroup, 32 by 32 (3015 rows of 2816 x 2816: 110, by 4 132; of 2816 x 256 27 and 58;
// 1024 of 2560 x 9728, 2560 workgroups, 127 and 115), then 64 by 32 (3015 of 17408 x
// 5120: 1100, 32 by 32 1155; 100,000 of 128 x 4096, bound by X, 281 and 505).
template <typename X, bool ZP, int G>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    const int64_t per = a.M / a.n_experts;  // rows an expert has
    if (a.n_experts > 1 && per <= 2) return few<X, ZP, G, 2, 2, 4>(w, a, s);
    if (a.n_experts > 1 && per <= 64) return few<X, ZP, G, 2, 2, 16>(w, a, s);
    if (per > 16) {
        const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, 32) : (a.M + 31) / 32;
        if (gm * ((w.N + 63) / 64) >= 5120) return few<X, ZP, G, 4, 1, 32>(w, a, s);
        if (gm * ((w.N + 31) / 32) >= 4096) return few<X, ZP, G, 2, 1, 32>(w, a, s);
        return few<X, ZP, G, 2, 4, 32>(w, a, s);
    }
    if (w.N <= 4096) return few<X, ZP, G, 1, 4, 16>(w, a, s);
    return few<X, ZP, G, 2, 4, 16>(w, a, s);
}

template <typename X, bool ZP>
hipError_t few(const G4Weights& w, const Rows& a, hipStream_t s) {
    if (w.group == 32) return few<X, ZP, 32>(w, a, s);
    if (w.group == 64) return few<X, ZP, 64>(w, a, s);
    return few<X, ZP, 128>(w, a, s);
}

// Tiles (of 16-bit results) or stream.  A workgroup of a tile goes through all of K
// by itself, so that few tiles leave CUs idle and take as long as many: 2560 x 9728 takes
// 92 us in tiles with 256 to 1024 rows, streamed 39 to 115, with 768 rows 95 and 92;
// 17408 x 5120 with 64 rows 56 and 38, with 128 51 and 65, with 256 70 and 110; 4096 x
// 4096 with 400 rows 41 and 42, with 600 42 and 58; 2816 x 2816 of 8 experts with 600 rows
// 41 and 40, with 1000 41 and 58.  With many experts the two meet near 1.5 million results
// too, whatever the rows of each, and near 0.7 million where sums are short: 704 x 2816 of
// 128 with 1024 rows 51 and 41, with 2048 53 and 54, with 4096 58 and 81; 2816 x 704 of 128
// with 128 rows 32 and 28, with 512 47 and 54 (the rule streams these), with 620 48 and 55,
// with 1024 50 and 61, with 2048 53 and 80; 1408 x 2816 of 64 with 620 rows 51 and 42, with
// 1024 53 and 51, with 2048 56 and 75; 14336 x 4096 of 8 with 64 rows 80 and 66, with 128
// 81 and 84, with 256 88 and 128; 4096 x 14336 of 8 with 256 171 and 146, with 512 174 and
// 222.  Narrow matrices leave most of a tile's
// 256 columns empty.  (fp32 results carry no rounded weights, and exact ones take the
// streamed form at any size: 3015 x 17408 x 5120 in 1.13 ms, 24,120 rows of 128 experts,
// 2816 x 704, in 326 us.)
template <typename X, typename T>
hipError_t matmul(const G4Weights& w, const Rows& a, hipStream_t s) {
    if (a.y_f32 || w.N < 128 || a.M * w.N < 1700000) return w.zeros ? few<X, true>(w, a, s) : few<X, false>(w, a, s);
    if (a.M / a.n_experts <= 64) return tile<T, 2, 2, 1>(w, a, s);
    return tile<T, 4, 2, 2>(w, a, s);
}

}  // namespace

hipError_t gqk_g4_matmul(const G4Weights& w, const void* X, int x_dtype, int64_t M, int64_t ldx, void* Y, int y_dtype,
                         int64_t ldy, int n_experts, const int32_t* offsets, hipStream_t s) {
    const Rows a{X, M, ldx, Y, ldy, y_dtype == gqd::DT_F32, n_experts, offsets};
    return x_dtype == gqd::DT_BF16 ? matmul<XBf16, Bf16>(w, a, s) : matmul<XF16, F16>(w, a, s);
}
