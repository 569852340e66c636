// gq_f8_matmul.hip -- products of block-scaled e4m3 activations and weights on
// the matrix cores (gfx950): gq_f8_matmul, and gq_f8_matmul_id for routed
// experts.
//
// Y[m][n] = sum_b xs[b][m] ws[n / 128][b] (sum_{k in b} X[m][k] W[n][k]): the
// sum over one group of 128 inputs is one 8-bit matrix instruction for a bf16
// Y, and four bf16 ones on the exactly widened operands for an fp32 Y
// (gq_f8_device.h: the 8-bit instruction keeps about 16 bits of a sum), which
// is then scaled into the fp32 accumulator.  W is
// the A operand and X the B operand, so a lane holds four consecutive columns
// of one row of Y: one activation scale per lane and tile, and adjacent stores.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "gq_f8_device.h"
#include "gq_f8_internal.h"
#include "gq_f8_stream.h"

using namespace gqf8;

namespace {

// ------------------------------------------------- slots by expert (plan) ----
// Workspace: header (int [0] = invalid ids, [1] = tiles), the tiles, each slot's
// expert (-1: invalid id), the slots by expert, the per-slot outputs of a
// weighted product.
struct WsLayout {
    int TM, max_tiles;
    size_t off_tile, off_expert, off_slot, off_out, total;
};

// A tile: rows slots, from position start of the slots by expert, of expert e.
struct alignas(16) TileEntry {
    int e, start, rows, unused;
};

// Slots of a tile, from what every product of a layer has in common.
int tile_rows(int64_t S, int n_experts);

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

WsLayout layout(int n_experts, int64_t S, int64_t N, int y_dtype, int weighted) {
    WsLayout L;
    L.TM = tile_rows(S, n_experts);
    // the worst case: every expert ends with a partial tile
    L.max_tiles = (int)(S / L.TM + (S < n_experts ? S : n_experts));
    L.off_tile = 256;
    L.off_expert = L.off_tile + up256(sizeof(TileEntry) * (size_t)L.max_tiles);
    L.off_slot = L.off_expert + up256(4 * (size_t)S);
    L.off_out = L.off_slot + up256(4 * (size_t)S);
    L.total = L.off_out + (weighted ? (size_t)S * (size_t)N * (y_dtype == gqd::DT_F32 ? 4 : 2) : 0);
    return L;
}

struct Table {
    int* hdr;
    TileEntry* tile;
    int *slot_e, *slot;
    int n_experts, S, top_k, per_slot;
    const int32_t* ids;  // given: the kernel makes the table itself (SMALL slots at most)
    int zero;            // it also zeroes the rows of invalid slots
};

constexpr int SMALL = 64;

constexpr int MAX_E = 4096;

// f(slot, id) for every slot, 4 * blockDim.x slots at a time; every thread of
// the workgroup makes the same number of calls (past the end: id INT_MAX, which
// no expert has).
template <typename F>
__device__ __forceinline__ void each_slot(const int32_t* __restrict__ ids, int S, F f) {
    auto at = [&](int s) {
        int4 v = make_int4(INT_MAX, INT_MAX, INT_MAX, INT_MAX);
        if (s + 4 <= S) {
            v = *reinterpret_cast<const int4*>(ids + s);  // (ids are 16-byte aligned)
        } else {
            if (s < S) v.x = ids[s];
            if (s + 1 < S) v.y = ids[s + 1];
            if (s + 2 < S) v.z = ids[s + 2];
        }
        return v;
    };
    constexpr int U = 8;  // loads on their way at once
    const int step = 4 * blockDim.x;
    for (int s0 = 0; s0 < S; s0 += U * step) {
        int4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u * step < S) v[u] = at(s0 + u * step + 4 * threadIdx.x);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u * step >= S) break;
            const int s = s0 + u * step + 4 * threadIdx.x;
            f(s, v[u].x);
            f(s + 1, v[u].y);
            f(s + 2, v[u].z);
            f(s + 3, v[u].w);
        }
    }
}

// Workgroup e < n_experts lists the slots of expert e (their order among
// themselves does not reach any result: each output row is computed on its
// own): once over the ids to count the smaller ones, once to place its own.
// The last workgroup counts the slots of every expert and cuts them into tiles
// of at most TM.  Where ids are invalid, the output rows (y) of their slots are
// zeroed by the wavefronts of all the others.  All read all ids, from the
// caches: one launch instead of a chain of counting, scanning and placing
// (24,120 slots of 128 experts: 9.7 us; 11 with four ids on their way, 60 with one).
template <typename TY>
__global__ __launch_bounds__(1024) void k_f8_plan(const int32_t* __restrict__ ids, int S, int n_experts, int TM,
                                                  int* __restrict__ hdr, TileEntry* __restrict__ tile,
                                                  int* __restrict__ slot_e, int* __restrict__ slot,
                                                  TY* __restrict__ y, int64_t N) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int e = blockIdx.x;
    if (e < n_experts) {
        __shared__ int n_less, n_here, any_bad;
        if (tid == 0) {
            n_less = 0;
            n_here = 0;
            any_bad = 0;
        }
        __syncthreads();
        int less = 0;
        bool bad = false;
        each_slot(ids, S, [&](int s, int id) {
            less += id >= 0 && id < e;
            bad |= s < S && (id < 0 || id >= n_experts);
        });
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) less += __shfl_xor(less, off, 64);
        if (lane == 0) atomicAdd(&n_less, less);
        if (bad) any_bad = 1;
        __syncthreads();
        const int base = n_less;
        each_slot(ids, S, [&](int s, int id) {
            const uint64_t vote = __ballot(id == e);
            if (vote == 0) return;  // (the same for the whole wavefront)
            int at = 0;
            if (lane == 0) at = atomicAdd(&n_here, __popcll(vote));
            at = __builtin_amdgcn_readfirstlane(at);
            if (id == e) slot[base + at + __popcll(vote & ((1ull << lane) - 1))] = s;
        });
        if (y && any_bad)
            each_slot(ids, S, [&](int s, int id) {
                uint64_t mine = __ballot(s < S && (id < 0 || id >= n_experts) && s % n_experts == e);
                for (; mine; mine &= mine - 1) {
                    const int64_t row = __builtin_amdgcn_readlane(s, __builtin_ctzll(mine));
                    for (int64_t n = lane; n < N; n += 64) store_as(y + row * N + n, 0.0f);
                }
            });
        return;
    }
    __shared__ int count[MAX_E];
    __shared__ int n_bad;
    if (tid == 0) n_bad = 0;
    for (int i = tid; i < n_experts; i += blockDim.x) count[i] = 0;
    __syncthreads();
    each_slot(ids, S, [&](int s, int id) {
        if (s >= S) return;
        const bool ok = id >= 0 && id < n_experts;
        slot_e[s] = ok ? id : -1;
        atomicAdd(ok ? &count[id] : &n_bad, 1);
    });
    __syncthreads();
    if (tid < 64) {
        // exclusive scans over the experts by one wavefront: each lane a run
        const int per = (n_experts + 63) / 64;
        const int lo = tid * per < n_experts ? tid * per : n_experts;
        const int hi = lo + per < n_experts ? lo + per : n_experts;
        int a = 0, b = 0;
        for (int i = lo; i < hi; ++i) {
            a += count[i];
            b += (count[i] + TM - 1) / TM;
        }
        int ia = a, ib = b;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int va = __shfl_up(ia, off, 64), vb = __shfl_up(ib, off, 64);
            if (tid >= off) {
                ia += va;
                ib += vb;
            }
        }
        int ra = ia - a, rb = ib - b;
        for (int i = lo; i < hi; ++i) {
            for (int c = 0; c < count[i]; c += TM)
                tile[rb++] = TileEntry{i, ra + c, count[i] - c < TM ? count[i] - c : TM, 0};
            ra += count[i];
        }
        if (tid == 63) {
            hdr[0] = n_bad;
            hdr[1] = ib;
        }
    }
}

// The expert and the slots [start, start + rows) of tile i; false where the
// table has no such tile.  Every field is clamped to its range.
__device__ __forceinline__ bool tile_of(const Table& t, int i, int TM, int& e, int& start, int& rows) {
    const TileEntry v = t.tile[i];
    if (i >= t.hdr[1]) return false;
    e = (unsigned)v.e < (unsigned)t.n_experts ? v.e : t.n_experts - 1;
    start = (unsigned)v.start < (unsigned)t.S ? v.start : t.S - 1;
    const int most = t.S - start < TM ? t.S - start : TM;
    rows = v.rows < most ? v.rows : most;
    return rows > 0;
}

// The same for a call with at most SMALL slots that is given ids: every
// wavefront finds tile i's slots itself, lane s standing for slot s, and the
// launch of a plan is saved (8 tokens x 8 of 128 experts: 5 of 22 us).  Slots of
// one expert find each other by a ballot for each bit of the id; the experts
// take their places in the order of their first slots.  own: the tile's slots.
// The first workgroup writes the header and each slot's expert, the first one of
// each tile its part of the table, for later calls without ids.
__device__ __forceinline__ bool tile_from_ids(const Table& t, int i, int TM, bool first_column, int& e, int& start,
                                              int& rows, int* own) {
    const int lane = threadIdx.x & 63;
    const bool lead = threadIdx.x < 64;
    const int id = lane < t.S ? t.ids[lane] : -1;
    const bool ok = id >= 0 && id < t.n_experts;
    const uint64_t valid = __ballot(ok);
    uint64_t same = valid;
#pragma unroll
    for (int b = 0; b < 12; ++b) {  // (n_experts <= 4096)
        const bool bit = (id >> b) & 1;
        const uint64_t m = __ballot(bit);
        same &= bit ? m : ~m;
    }
    const int count = __popcll(same), rank = __popcll(same & ((1ull << lane) - 1));
    const bool head = ok && rank == 0;
    // slots (low half) and tiles of the experts up to this lane's
    const int n = head ? count | (((count + TM - 1) / TM) << 16) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(incl, off, 64);
        if (lane >= off) incl += v;
    }
    const int before = incl - n, tb = before >> 16;
    if (i == 0 && first_column && lead) {
        if (lane < t.S) t.slot_e[lane] = ok ? id : -1;
        if (lane == 63) {
            t.hdr[0] = t.S - __popcll(valid);
            t.hdr[1] = incl >> 16;
        }
    }
    const uint64_t hit = __ballot(head && tb <= i && i < tb + (n >> 16));
    if (hit == 0) return false;
    const int l = __builtin_ctzll(hit);
    e = __builtin_amdgcn_readlane(id, l);
    const int c = i - __builtin_amdgcn_readlane(tb, l), left = __builtin_amdgcn_readlane(count, l) - c * TM;
    start = (__builtin_amdgcn_readlane(before, l) & 0xffff) + c * TM;
    rows = left < TM ? left : TM;
    const int place = rank - c * TM;
    if (ok && id == e && place >= 0 && place < rows) {
        own[place] = lane;
        if (first_column && lead) t.slot[start + place] = lane;
    }
    if (first_column && threadIdx.x == 0) t.tile[i] = TileEntry{e, start, rows, 0};
    return true;
}

// ------------------------------------------------------- many rows (tiles) ----
// Order of the tiles: workgroups go to the 8 XCDs in turn, so XCD x takes a run
// of neighbouring tiles (each XCD has an L2 of its own), and a run walks the
// row tiles of one column of tiles first: 32 CUs then share a few panels of W
// and all (at most G) panels of X.
__device__ __forceinline__ int xcd_order(int id, int total) {
    const int x = id & 7, q = total >> 3, r = total & 7;
    return x * q + (x < r ? x : r) + (id >> 3);
}

// BM rows of X by BN rows of W; WM x WN wavefronts of (BM / WM) x (BN / WN).
// Both tiles of a 128-input block go to LDS by global-to-LDS copies, NB blocks
// ahead, in rows of 128 bytes whose 16-byte chunks are swizzled so that
// operand reads cover all banks; the block's activation scales come along.
// One barrier a block.
//
// Operand row a of the MFMA tiles 2 p and 2 p + 1 is the tile's column 32 p +
// 8 (a / 4) + a % 4 (+ 4 for the second), so that a lane ends up with eight
// neighbouring columns of one row of Y: 16-byte stores, 64-byte runs.
//
// What bounds it (256 x 256, bf16 result; timing variants of 3015 x 16384 x
// 5120, three whole rounds, 248 us): the copies alone take 228 us (8.8 TB/s from
// the L2s; 150 us if all of them hit), the products with the scaling 192 us,
// the matrix instructions alone 154 us.  Reading each line ahead into the L2
// cost more than it gave (262-285 us).  The L2s fetch 4.4 times the operands'
// bytes for 3015 x 17408 x 5120.  Measured: that in 262-271
// us (1.98-2.05 PFLOP/s; a vendor's product with one scale for each operand
// takes 268-276 us), 8100 x 8192 x 8192 in 482 us (2.26 PFLOP/s).
//
// FAR (routed): X may span more than 2^31 bytes, so its rows are addressed by
// pointers, two registers each, instead of offsets.
template <int BM, int BN, int WM, int WN, int NB, typename TY, bool ROUTED, bool FAR>
struct Tile {
    static constexpr int WV = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
    static constexpr int XI = BM / 8 / WV, WI = BN / 8 / WV;  // copies of a wavefront and block
    static constexpr int SX = (BM + BN) * BLK, STAGE = SX + WV * 256;
    static constexpr int LOADS = XI + WI + 1;
    // (with the 256 x 256 tile's registers the longer loop does not fit)
    static constexpr bool MANY = ROUTED && BM < 256;
    static_assert(BM % (8 * WV) == 0 && BN % (8 * WV) == 0 && WV > BM / 64 && BN / WN <= BLK, "tile shape");

    // swizzle of W's rows: (r / 2 % 2, r / 8 % 4), the rows of one operand read
    static __device__ __forceinline__ int wswz(int r) { return ((r >> 1) & 1) | (((r >> 3) & 3) << 1); }

    // rows of X from m0 (routed: the slots from `start`) by `count` tiles of
    // columns from n0, one after another without a gap: the copies run NB blocks
    // ahead of the products, over the end of a tile into the next (MANY).
    static __device__ __forceinline__ void run(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                               int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                               const float* __restrict__ xs, int64_t ldx, int64_t xs_ld,
                                               TY* __restrict__ Y, int64_t ldy, int64_t m0, int64_t n0, int rows,
                                               int start, int count, const Table& t, uint8_t* smem) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int fr = lane & 15, fq = lane >> 4;
        const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
        const int KB = (int)((K + BLK - 1) / BLK);
        auto slot_of = [&](int i) -> int64_t {
            const unsigned s = (unsigned)t.slot[start + (i < rows ? i : rows - 1)];
            return s < (unsigned)t.S ? (int64_t)s : t.S - 1;
        };
        auto routed_row = [&](int i) -> int64_t { return t.per_slot ? slot_of(i) : slot_of(i) / t.top_k; };

        // Copies.  Wavefront w brings rows 8 (w + WV u) .. + 7 of either tile; the
        // chunk of row r that a lane copies is the one its position holds.
        const int lr = 8 * wave + (lane >> 3);
        static_assert(WV % 4 == 0, "the swizzle of a lane's rows is the same for all of its copies");
        const uint32_t xchunk = 16u * (uint32_t)((lane & 7) ^ ((lr >> 1) & 7));
        const uint32_t wchunk = 16u * (uint32_t)((lane & 7) ^ wswz(lr));
        const uint32_t woff = (uint32_t)(lr * K) + wchunk;
        // X: one offset and a common step, or (routed) each copy's own row
        uint32_t xoff[ROUTED ? XI : 1];
        const uint8_t* xp[FAR ? XI : 1];
#pragma unroll
        for (int u = 0; u < (ROUTED ? XI : 1); ++u) {
            if constexpr (FAR) xp[u] = X + routed_row(lr + 8 * WV * u) * ldx;
            else if constexpr (ROUTED) xoff[u] = (uint32_t)(routed_row(lr + 8 * WV * u) * ldx) + xchunk;
            else xoff[u] = (uint32_t)(lr * ldx) + xchunk;
        }
        const int64_t x_rows = t.per_slot ? t.S : t.S / (t.top_k > 0 ? t.top_k : 1);
        const Rsrc xr = make_rsrc(X, ROUTED && !FAR ? x_rows * ldx : 0);
        // Rows 8 WV u and on of `rows` rows of `width` bytes from p: each copy has a
        // resource of its own, so that no row past the last one is read whether or
        // not the range check counts the scalar offset (an offset of k is within
        // the lane's row).
        auto rows_from = [](const uint8_t* p, int u, int rows, int64_t width) {
            const int n = rows - 8 * WV * u;
            return make_rsrc(p + 8 * WV * u * width, (n > 0 ? n : 0) * (int)width);
        };
        // one copy of 64 scales: wavefronts below BM / 64 those of X, the others
        // W's (lane w: of wavefront w's columns), from sbase[slane + ck * sstep];
        // a tile further (routed), W's lie snext on, as far as the last row of blocks
        static_assert(!ROUTED || BN % BLK == 0, "whole blocks of columns");
        const bool xwave = wave < BM / 64;
        const float* sbase = xwave ? xs : wsc;
        const int64_t sstep = xwave ? xs_ld : 1;
        const int slast = xwave ? INT_MAX : (int)((N - 1) / BLK) * KB, snext = xwave ? 0 : BN / BLK * KB;
        int slane;
        if (xwave) {
            const int i = 64 * wave + lane;
            if constexpr (ROUTED) slane = (int)routed_row(i);
            else slane = (int)m0 + (i < rows ? i : rows - 1);
        } else {
            const int64_t n = n0 + (lane % WV / WM) * (BN / WN);
            slane = (int)((n < N ? n : N - 1) / BLK) * KB;
        }
        // what the copies read next: block ck of the columns from cn, into buffer cg
        int ck = 0, cg = 0;
        int64_t cn = n0;
        const int64_t n_end = n0 + (int64_t)count * BN;
        auto load = [&]() {
            uint8_t* d = smem + cg * STAGE;
            cg = cg + 1 == NB ? 0 : cg + 1;
            const int k = ck * BLK;
            const int left = (int)K - k, wleft = cn < n_end ? left : 0;  // (W past the last tile: zeros)
            const int w_rows = N - cn < BN ? (int)(N - cn) : BN;
            const uint32_t wo = within(woff, (int)wchunk, wleft);
            // (FAR: past K the row's first chunk, times zeros)
            const int xk = k + ((int)xchunk < left ? (int)xchunk : -k);
#pragma unroll
            for (int u = 0; u < XI; ++u) {
                uint8_t* l = d + (wave + WV * u) * 1024;
                if constexpr (FAR) copy16(xp[u] + xk, l);
                else if constexpr (ROUTED) copy16(xr, within(xoff[u], (int)xchunk, left), l, (uint32_t)k);
                else copy16(rows_from(X + m0 * ldx, u, rows, ldx), within(xoff[0], (int)xchunk, left), l, (uint32_t)k);
            }
#pragma unroll
            for (int u = 0; u < WI; ++u)
                copy16(rows_from(W + cn * K, u, w_rows, K), wo, d + BM * BLK + (wave + WV * u) * 1024, (uint32_t)k);
            copy4(sbase + (slane + (ck < KB ? ck : KB - 1) * sstep), d + SX + wave * 256);
            ++ck;
            if constexpr (MANY) {
                const bool wrap = ck == KB;  // (no branch: it would split what is scheduled together)
                ck = wrap ? 0 : ck;
                cn += wrap ? BN : 0;
                slane += wrap ? snext : 0;
                slane = slane < slast ? slane : slast;
            }
        };
        f32x4 acc[NT][MT];
        auto clear = [&]() {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{};
        };
        const bool vec = (ldy & (16 / (int)sizeof(TY) - 1)) == 0;
        int y_slot[ROUTED ? MT : 1];
        if constexpr (ROUTED) {
#pragma unroll
            for (int j = 0; j < MT; ++j) y_slot[j] = (int)slot_of(wm + 16 * j + fr);
        }
        auto store = [&]() {
            int l = lane;  // opaque: otherwise all the addresses are computed ahead of the loop, and spilled
            __asm__ volatile("" : "+v"(l));
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int row = wm + 16 * j + (l & 15);
                if (row >= rows) continue;
                TY* y = Y + (ROUTED ? y_slot[ROUTED ? j : 0] : m0 + row) * ldy;
#pragma unroll
                for (int i = 0; i < NT; i += 2)
                    store8(y, n0 + wn + 16 * i + 8 * (l >> 4), N, vec, acc[i][j], acc[i + 1][j]);
            }
        };
        clear();
        if (KB == 0) {
            for (int i = 0; i < count; ++i, n0 += BN) store();
            return;
        }

        // Operands.  16-byte positions of this lane's two chunks of an operand row: of X in rows 16 j + fr, of W in
        // rows 32 (i / 2) + 8 (fr / 4) + 4 (i % 2) + fr % 4 (whose swizzle is the same for every i).
        const int p0 = pos128(fr, fq), p1 = pos128(fr, 4 + fq);
        const int ar = 8 * (fr >> 2) + (fr & 3), w0 = ar * 8 + (fq ^ wswz(ar)), w1 = ar * 8 + ((4 + fq) ^ wswz(ar));
        auto w_operand = [&](int g, int i) {
            const u32x4* d = reinterpret_cast<const u32x4*>(smem + g * STAGE + (BM + wn) * BLK);
            const int at = 256 * (i >> 1) + 32 * (i & 1);
            return join(d[at + w0], d[at + w1]);
        };
        auto x_operand = [&](int g, int j) {
            const u32x4* d = reinterpret_cast<const u32x4*>(smem + g * STAGE + wm * BLK);
            return join(d[128 * j + p0], d[128 * j + p1]);
        };
        auto scales = [&](int g, float (&s)[MT]) {
            const float* d = reinterpret_cast<const float*>(smem + g * STAGE + SX);
            const float s_w = d[(BM / 64) * 64 + wave];
#pragma unroll
            for (int j = 0; j < MT; ++j) s[j] = s_w * d[wm + 16 * j + fr];
        };
        auto product = [&](i32x8 a, const i32x8 (&x)[MT], f32x4 (&p)[MT]) {
            if constexpr (sizeof(TY) == 4) {
                const Wide aw = widen(a);
#pragma unroll
                for (int j = 0; j < MT; ++j) p[j] = mfma16(aw, widen(x[j]));
            } else {
#pragma unroll
                for (int j = 0; j < MT; ++j) p[j] = mfma8(a, x[j]);
            }
        };
        auto add = [&](int i, const f32x4 (&p)[MT], const float (&s)[MT]) {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[j][r], s[j], acc[i][j][r]);
        };
        // A block, whose operands x, first a and scales s are in registers: each
        // W operand is read while the one before it is multiplied, the last before
        // the barrier.  The barrier then says two things: the next block has landed
        // for everyone, and nobody needs this block's buffer, into which the one NB
        // ahead is sent; the next block's first operands are read while the last
        // products run.
#pragma unroll
        for (int b = 0; b < NB; ++b) load();
        wait_copies<(NB - 1) * LOADS>();
        gqd::lds_barrier();
        if (ROUTED && wm >= rows) {
            // nothing of this wavefront's rows is used: it brings data only
            for (int64_t b = 0; b < (int64_t)count * KB; ++b) {
                wait_copies<(NB - 2) * LOADS>();
                gqd::lds_barrier();
                load();
            }
            wait_copies<0>();
            return;
        }
        i32x8 x[MT], a = w_operand(0, 0);
        float s[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) x[j] = x_operand(0, j);
        scales(0, s);
        int g = 0;
        for (int tile = 0;;) {
            int kb = 0;
            do {
                f32x4 p[MT];
#pragma unroll
                for (int i = 0; i < NT - 1; ++i) {
                    __builtin_amdgcn_sched_barrier(0);
                    const i32x8 next = w_operand(g, i + 1);
                    f32x4 q[MT];
                    product(a, x, q);
                    if (i > 0) add(i - 1, p, s);
#pragma unroll
                    for (int j = 0; j < MT; ++j) p[j] = q[j];
                    a = next;
                    if constexpr (sizeof(TY) == 2) {
                        // the reads after the first product: at its wait nothing younger is outstanding
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // MFMA
                            if (j == 0) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
                            if (i > 0) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // VALU
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                wait_copies<(NB - 2) * LOADS>();
                gqd::lds_barrier();
                load();
                g = g + 1 == NB ? 0 : g + 1;
                f32x4 q[MT];
                product(a, x, q);
                __builtin_amdgcn_sched_barrier(0);  // (x, a are read into their own registers again)
                add(NT - 2, p, s);
                a = w_operand(g, 0);
#pragma unroll
                for (int j = 0; j < MT; ++j) x[j] = x_operand(g, j);
                add(NT - 1, q, s);
                scales(g, s);
            } while (++kb < KB);
            store();
            if (!MANY || ++tile == count) break;
            clear();
            n0 += BN;
        }
        wait_copies<0>();
    }
};

// Row tiles of a band: 4 by 8 tiles are what 32 CUs of an XCD work on at once,
// with the least to read (3015 x 17408 x 5120: 266 us; 12: 272, 2: 274 us).
constexpr int BAND = 4;

// Dense.  Workgroups from n_full on take quarters of the tiles from n_full on
// (QUARTERS): the last, partial round of 256 x 256 tiles would take as long as a
// whole one on a part of the CUs.
template <int BM, int BN, int WM, int WN, int NB, typename TY, bool QUARTERS>
__global__ __launch_bounds__(64 * WM * WN) void k_f8_tile(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                                          int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                                          const float* __restrict__ xs, int64_t M, int64_t ldx,
                                                          int64_t xs_ld, TY* __restrict__ Y, int64_t ldy, int gm,
                                                          int gn, int n_full) {
    using T = Tile<BM, BN, WM, WN, NB, TY, false, false>;
    constexpr int D = QUARTERS ? 2 : 1;
    using Q = Tile<BM / D, BN / D, WM, WN, NB * D, TY, false, false>;
    constexpr int LDS = NB * T::STAGE, QLDS = NB * D * Q::STAGE;
    __shared__ __align__(16) uint8_t smem[LDS > QLDS ? LDS : QLDS];
    const Table none{};
    auto place = [&](int id, int64_t& m0, int64_t& n0) {
        // bands of at most BAND row tiles, each walked column of tiles by column
        const int bands = (gm + BAND - 1) / BAND, h = (gm + bands - 1) / bands;
        const int band = id / (h * gn), hb = gm - band * h < h ? gm - band * h : h;
        const int c = id - band * h * gn;
        m0 = (int64_t)(band * h + c % hb) * BM;
        n0 = (int64_t)(c / hb) * BN;
    };
    int64_t m0, n0;
    if constexpr (QUARTERS) {
        const int q = (int)blockIdx.x - n_full;
        if (q >= 0) {
            place(n_full + (q >> 2), m0, n0);
            m0 += (q & 1) * (BM / 2);
            n0 += (q >> 1 & 1) * (BN / 2);
            if (m0 >= M || n0 >= N) return;
            const int64_t left = M - m0;
            Q::run(W, wsc, N, K, X, xs, ldx, xs_ld, Y, ldy, m0, n0, (int)(left < BM / 2 ? left : BM / 2), 0, 1, none,
                   smem);
            return;
        }
    }
    place(xcd_order(blockIdx.x, n_full), m0, n0);
    T::run(W, wsc, N, K, X, xs, ldx, xs_ld, Y, ldy, m0, n0, (int)(M - m0 < BM ? M - m0 : BM), 0, 1, none, smem);
}

// Routed: the rows of table tile blockIdx.x / split and the blockIdx.x % split-th
// share of the gn columns of tiles.
template <int BM, int BN, int WM, int WN, int NB, typename TY, bool FAR>
__global__ __launch_bounds__(64 * WM * WN) void k_f8_tile_id(const uint8_t* __restrict__ W,
                                                             const float* __restrict__ wsc, int64_t N, int64_t K,
                                                             const uint8_t* __restrict__ X,
                                                             const float* __restrict__ xs, int64_t ldx, int64_t xs_ld,
                                                             TY* __restrict__ Y, int gm, int gn, int split, Table t) {
    using T = Tile<BM, BN, WM, WN, NB, TY, true, FAR>;
    __shared__ __align__(16) uint8_t smem[NB * T::STAGE];
    // (the grid is sized for the most tiles there can be: only the real ones are dealt out to the XCDs)
    const int tiles = t.hdr[1], real = (tiles < gm ? tiles : gm) * split;
    if ((int)blockIdx.x >= real) return;
    const int id = xcd_order(blockIdx.x, real), tm = id / split, part = id % split;
    const int first = (int)((int64_t)gn * part / split), end = (int)((int64_t)gn * (part + 1) / split);
    int e, start, rows;
    if (!tile_of(t, tm, BM, e, start, rows)) return;
    W += (int64_t)e * N * K;
    wsc += (int64_t)e * ((N + BLK - 1) / BLK) * ((K + BLK - 1) / BLK);
    T::run(W, wsc, N, K, X, xs, ldx, xs_ld, Y, N, 0, (int64_t)first * BN, rows, start, end - first, t, smem);
}

// Routed, bf16 results, short rows (at most KB <= 6 blocks of 128): a wavefront
// keeps its 32 rows of X in registers, for all of K, and only W goes through LDS,
// in panels of 32 columns and all of K.  Beside half the copies, a panel is one
// piece of memory whose lines are read at one time (blocks of 128 inputs of rows
// of 704 bytes share lines).  The panels are copied two ahead, block by block,
// their rows in the operands' order (see Tile: a lane ends up with eight
// neighbouring columns), the chunks swizzled as there.  A panel's results are
// stored behind the next barrier, ahead of the next copies, so that no wait is for
// a store just made.
// 3015 x 8 slots of 128 experts, 2816 x 704: 117 us in the median of a trace, 113
// at least (128 x 128 tiles: 148 us); of these 113, 82 are left without the copies,
// 90 without the stores, and 22 are two starts one after the other.  It fetches 1.2
// times its operands' bytes.  X through LDS in whole lines starts sooner but holds
// the panels up (146 against 147 us a call, other shapes 8% less to 6% more); whole
// rows of a panel one after another, of odd stride, have bank conflicts (147 against
// 146 us).  6 blocks take 208 registers and 72 KB of LDS, so that two workgroups run
// on a CU; 8 would take 96 KB and more than 256 registers.
constexpr int PANELS = 3;

template <int KB, int WV>
__global__ __launch_bounds__(64 * WV, 2) void k_f8_short_id(const uint8_t* __restrict__ W,
                                                            const float* __restrict__ wsc, int64_t N, int64_t K,
                                                            const uint8_t* __restrict__ X,
                                                            const float* __restrict__ xs, int64_t ldx, int64_t xs_ld,
                                                            uint16_t* __restrict__ Y, int gm, int gn, int split,
                                                            Table t) {
    // copies of a panel, and of a wavefront
    constexpr int NI = 4 * KB, CI = NI / WV;
    static_assert(NI % WV == 0, "whole copies");
    __shared__ __align__(16) uint8_t smem[PANELS * NI * 1024];
    const int tiles = t.hdr[1], real = (tiles < gm ? tiles : gm) * split;
    if ((int)blockIdx.x >= real) return;
    const int id = xcd_order(blockIdx.x, real), tm = id / split, part = id % split;
    const int first = (int)((int64_t)gn * part / split), end = (int)((int64_t)gn * (part + 1) / split);
    int e, start, rows;
    if (!tile_of(t, tm, 32 * WV, e, start, rows)) return;
    const int kbs = (int)((K + BLK - 1) / BLK);
    W += (int64_t)e * N * K;
    wsc += (int64_t)e * ((N + BLK - 1) / BLK) * kbs;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4, wm = 32 * wave;
    auto slot_of = [&](int i) -> int64_t {
        const unsigned s = (unsigned)t.slot[start + (i < rows ? i : rows - 1)];
        return s < (unsigned)t.S ? (int64_t)s : t.S - 1;
    };

    // copy i of a panel: of block i / 4 the rows 8 (i % 4) .. + 7, in the operands' order
    uint32_t off[CI];
#pragma unroll
    for (int u = 0; u < CI; ++u) {
        const int i = wave + WV * u, r = 8 * (i & 3) + (lane >> 3), c = 8 * (i >> 2) + ((lane & 7) ^ ((r >> 1) & 7));
        const int row = 8 * ((r & 15) >> 2) + 4 * (r >> 4) + (r & 3);
        off[u] = 16 * c < K ? (uint32_t)(row * K + 16 * c) : NOWHERE;
    }
    auto load = [&](int panel, int buf) {
        const int64_t n = (int64_t)panel * 32;
        const Rsrc r = make_rsrc(W + n * K, panel < end ? (N - n < 32 ? N - n : 32) * K : 0);
#pragma unroll
        for (int u = 0; u < CI; ++u) copy16(r, off[u], smem + 1024 * (buf * NI + wave + WV * u));
    };
    load(first, 0);
    load(first + 1, 1);

    int64_t x_row[2];
    uint16_t* y_row[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t s = slot_of(wm + 16 * j + fr);
        x_row[j] = t.per_slot ? s : s / t.top_k;
        y_row[j] = Y + s * N;
    }
    const Rsrc xr = make_rsrc(X, (t.per_slot ? t.S : t.S / t.top_k) * ldx);
    i32x8 x[KB][2];
    float sx[KB][2], f[KB][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = kb * BLK + 16 * fq;
            const uint32_t o = (uint32_t)(x_row[j] * ldx) + k;
            x[kb][j] = join(bld16(xr, within(o, k, (int)K)), bld16(xr, within(o + 64, k + 64, (int)K)));
            sx[kb][j] = kb < kbs ? xs[kb * xs_ld + x_row[j]] : 0.0f;
        }
    const bool idle = wm >= rows, vec = (N & 7) == 0;  // (idle: none of this wavefront's rows is used)
    const int at0 = pos128(fr, fq), at1 = pos128(fr, 4 + fq);  // (16 rows further: 128 positions)
    f32x4 acc[2][2];
    auto store = [&](int panel) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (wm + 16 * j + fr < rows) store8(y_row[j], (int64_t)panel * 32 + 8 * fq, N, vec, acc[0][j], acc[1][j]);
    };
    int buf = 0;
    for (int p = first; p < end; ++p) {
        wait_copies<CI>();
        gqd::lds_barrier();
        if (p > first) store(p - 1);
        load(p + 2, buf == 0 ? 2 : buf - 1);
        if (!idle) {
            if (p == first || (p & 3) == 0) {
                const float* s = wsc + (int64_t)(p >> 2) * kbs;
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const float w = s[kb < kbs ? kb : 0];
#pragma unroll
                    for (int j = 0; j < 2; ++j) f[kb][j] = w * sx[kb][j];
                }
            }
            const u32x4* d = reinterpret_cast<const u32x4*>(smem + buf * (NI * 1024));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const i32x8 a[2] = {join(d[256 * kb + at0], d[256 * kb + at1]),
                                    join(d[256 * kb + 128 + at0], d[256 * kb + 128 + at1])};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f32x4 q = mfma8(a[i], x[kb][j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(q[r], f[kb][j], acc[i][j][r]);
                    }
            }
        }
        buf = buf == 2 ? 0 : buf + 1;
    }
    if (end > first) store(end - 1);
    wait_copies<0>();
}

// A few rows: the stream kernel, 16 MT rows of X and 16 NT of W a workgroup.
template <int MT, int NT, int WV, typename TY, bool ROUTED>
__global__ __launch_bounds__(64 * WV) void k_f8_stream(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                                       int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                                       const float* __restrict__ xs, int64_t M, int64_t ldx,
                                                       int64_t xs_ld, TY* __restrict__ Y, int64_t ldy, Table t) {
    constexpr int RING = WV * Stream<MT, NT, X_E4M3, 16 * MT>::BYTES, JOIN = WV * NT * MT * 1024;
    __shared__ __align__(16) uint8_t smem[RING > JOIN ? RING : JOIN];
    const int tn = blockIdx.x, tm = blockIdx.y;
    int e = 0, start = 0, rows;
    __shared__ int own[ROUTED ? 16 * MT : 1];
    const int* slots = nullptr;
    if constexpr (ROUTED) {
        if (t.ids) {
            if (tm == 0 && t.zero && threadIdx.x < 64) {
                // this workgroup's columns of the invalid slots' rows
                const int id = threadIdx.x < t.S ? t.ids[threadIdx.x] : 0;
                const int64_t n = (int64_t)tn * (16 * NT) + threadIdx.x;
                for (uint64_t bad = __ballot(id < 0 || id >= t.n_experts); bad; bad &= bad - 1)
                    if (threadIdx.x < 16 * NT && n < N) store_as(Y + __builtin_ctzll(bad) * N + n, 0.0f);
            }
            if (!tile_from_ids(t, tm, 16 * MT, tn == 0, e, start, rows, own)) return;
            __syncthreads();
            slots = own;
        } else {
            if (!tile_of(t, tm, 16 * MT, e, start, rows)) return;
            slots = t.slot + start;
        }
        W += (int64_t)e * N * K;
        wsc += (int64_t)e * ((N + BLK - 1) / BLK) * ((K + BLK - 1) / BLK);
    } else {
        const int64_t left = M - (int64_t)tm * (16 * MT);
        rows = (int)(left < 16 * MT ? left : 16 * MT);
    }
    auto row_of = [&](int i) -> int64_t {
        const int c = i < rows ? i : rows - 1;
        if constexpr (ROUTED) {
            const unsigned s = (unsigned)slots[c];
            return s < (unsigned)t.S ? (int64_t)s : t.S - 1;
        } else {
            return (int64_t)tm * (16 * MT) + c;
        }
    };
    stream_tile<MT, NT, WV, X_E4M3, 16 * MT, TY>(
        W, wsc, (int64_t)tn * (16 * NT), N, K, X, xs, ldx, xs_ld, rows, (ldy & 3) == 0,
        [&](int i) { return ROUTED && !t.per_slot ? row_of(i) / t.top_k : row_of(i); },
        [&](int i) { return Y + row_of(i) * ldy; }, smem);
}

// y[t][n] = sum_j rw[t][j] slot[t][j][n], j in increasing order, slots of
// invalid ids left out.  Bound by the slots' bytes; a workgroup takes a token
// and 256 V columns of it, V of them a thread (16 bytes, where N allows): 3015 x
// 8 slots of 2816 bf16 in 23 us (6.6 TB/s, part of it still in the caches; 125
// us one element a thread).  Slots are held in the result's type: with bf16
// each is rounded once before the sum, which adds to the result's own rounding
// (together 1.41 times its error: 0.0023 against 0.0017 of the result's size), and
// halves the bytes that bound this.
template <typename TY, int V>
__global__ __launch_bounds__(256) void k_f8_combine(const TY* __restrict__ slots, const int* __restrict__ slot_e,
                                                    const float* __restrict__ rw, int top_k, int64_t N,
                                                    TY* __restrict__ y) {
    const int64_t t = blockIdx.x;
    for (int64_t n = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V; n < N; n += (int64_t)gridDim.y * (256 * V)) {
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.0f;
#pragma unroll 4
        for (int j = 0; j < top_k; ++j) {
            const int64_t s = t * top_k + j;
            const float w = rw[s];
            const bool ok = slot_e[s] >= 0;  // (otherwise nobody wrote the row)
            const TY* p = slots + s * N + n;
            if constexpr (V == 1) {
                const float v = sizeof(TY) == 4 ? (float)*p : gqd::bf2f((uint16_t)*p);
                sum[0] = ok ? __builtin_fmaf(w, v, sum[0]) : sum[0];
            } else if constexpr (sizeof(TY) == 4) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] = ok ? __builtin_fmaf(w, v[i], sum[i]) : sum[i];
            } else {
                const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = __builtin_bit_cast(float, i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
                    sum[i] = ok ? __builtin_fmaf(w, f, sum[i]) : sum[i];
                }
            }
        }
        if constexpr (V == 1) {
            store_as(y + t * N + n, sum[0]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                store4(y + t * N, n + i, N, true, f32x4{sum[i], sum[i + 1], sum[i + 2], sum[i + 3]});
        }
    }
}

template <int V, typename TY>
hipError_t combine(const TY* slots, const int* slot_e, const float* rw, int n_tokens, int top_k, int64_t N, TY* y,
                   hipStream_t s) {
    const int64_t gx = (N + 256 * V - 1) / (256 * V);
    const dim3 grid((unsigned)n_tokens, (unsigned)(gx < 65535 ? gx : 65535));
    hipLaunchKernelGGL((k_f8_combine<TY, V>), grid, dim3(256), 0, s, slots, slot_e, rw, top_k, N, y);
    return hipGetLastError();
}

// One call's operands.
template <typename TY>
struct Call {
    const uint8_t* W;
    const float* wsc;
    int64_t N, K;
    const uint8_t* X;
    const float* xs;
    int64_t M, ldx, xs_ld;  // M: rows of X, or slots
    TY* Y;
    int64_t ldy;
    Table t;
    hipStream_t s;
};

// gm: tiles of rows (of slots: the most there can be)
template <int MT, int NT, int WV, bool ROUTED, typename TY>
hipError_t stream(const Call<TY>& c, int64_t gm) {
    const int64_t gn = (c.N + 16 * NT - 1) / (16 * NT);
    // (routed: at most 8 slots an expert, 6144 tiles; dense: few rows)
    if (!grid_ok(gn, 64 * WV) || gm > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_f8_stream<MT, NT, WV, TY, ROUTED>), dim3((unsigned)gn, (unsigned)gm), dim3(64 * WV), 0, c.s,
                       c.W, c.wsc, c.N, c.K, c.X, c.xs, c.M, c.ldx, c.xs_ld, c.Y, c.ldy, c.t);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NB, bool QUARTERS, typename TY>
hipError_t tile(const Call<TY>& c) {
    const int64_t gm = (c.M + BM - 1) / BM, gn = (c.N + BN - 1) / BN, tiles = gm * gn;
    const int64_t cus = gqk_cu_count(), tail = tiles % cus;
    // quarters of the last round's tiles where they fit in one round themselves
    const int64_t n_full = QUARTERS && tiles > cus && 4 * tail <= cus ? tiles - tail : tiles;
    const int64_t grid = n_full + 4 * (tiles - n_full);
    if (!grid_ok(grid, 64 * WM * WN)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_f8_tile<BM, BN, WM, WN, NB, TY, QUARTERS>), dim3((unsigned)grid), dim3(64 * WM * WN), 0, c.s,
                       c.W, c.wsc, c.N, c.K, c.X, c.xs, c.M, c.ldx, c.xs_ld, c.Y, c.ldy, (int)gm, (int)gn,
                       (int)n_full);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NB, bool FAR, typename TY>
hipError_t tile_id(const Call<TY>& c, int64_t gm) {
    // two tiles of columns a workgroup (one with 256 rows): the second one's copies hide the first one's end;
    // more where a launch would have too many workgroups (at most 20,480 tiles of slots: at least one each)
    const int64_t gn = (c.N + BN - 1) / BN, most = (((int64_t)1 << 32) - 1) / (64 * WM * WN) / gm;
    const int64_t split = BM < 256 ? ((gn + 1) / 2 < most ? (gn + 1) / 2 : most) : gn;
    hipLaunchKernelGGL((k_f8_tile_id<BM, BN, WM, WN, NB, TY, FAR>), dim3((unsigned)(gm * split)), dim3(64 * WM * WN),
                       0, c.s, c.W, c.wsc, c.N, c.K, c.X, c.xs, c.ldx, c.xs_ld, c.Y, (int)gm, (int)gn, (int)split,
                       c.t);
    return hipGetLastError();
}

// n_tiles: the tiles that are likely.  About 4 workgroups of four wavefronts a CU
// (two run at once), or one of eight; each loads its rows of X first, so none has
// fewer than 3 panels (weighted 2816 x 704, 188 slots for each of 128 experts: 154,
// 146 and 146 us with 500, 1000 and 2000 workgroups; 2816 x 768, 754 for each of
// 16: 85, 61 and 64 us with 130, 260 and 510 of eight; 704 x 640, 377 for each of
// 16: 23.4 and 24.0 us with at least 3 and 6 panels each).
template <int KB, int WV>
hipError_t short_id(const Call<uint16_t>& c, int64_t gm, int64_t n_tiles) {
    const int64_t gn = (c.N + 31) / 32, groups = gqk_cu_count() * (WV == 4 ? 4 : 1);
    const int64_t want = groups > n_tiles ? groups / n_tiles : 1, most = (gn + 2) / 3;
    const int64_t split = want < most ? want : most;
    hipLaunchKernelGGL((k_f8_short_id<KB, WV>), dim3((unsigned)(gm * split)), dim3(64 * WV), 0, c.s, c.W, c.wsc, c.N,
                       c.K, c.X, c.xs, c.ldx, c.xs_ld, c.Y, (int)gm, (int)gn, (int)split, c.t);
    return hipGetLastError();
}

// (K padded to 2, 4 or 6 blocks: constants, so that the operands are read ahead)
template <int WV>
hipError_t short_id(const Call<uint16_t>& c, int64_t gm, int64_t n_tiles) {
    if (c.K > 4 * BLK) return short_id<6, WV>(c, gm, n_tiles);
    if (c.K > 2 * BLK) return short_id<4, WV>(c, gm, n_tiles);
    return short_id<2, WV>(c, gm, n_tiles);
}


// Which kernel: measured at N x K of 1024 x 2560, 5120 x 5120, 2560 x 9728 and
// 17408 x 5120, 16 to 2048 rows, and at N of 20,480 to 151,936, 17 to 769 rows.
// What decides is how many tiles there are for the CUs.  Few 64 x 128 tiles: the
// stream kernel, which splits K (256 rows of 2560 x 9728: 15.4 us against 30.6 us
// in tiles).  Up to one a CU: those tiles, eight wavefronts each and four blocks
// ahead (2048 rows of 1024 x 2560: 11.6 against 14.6 us two blocks ahead, 19.6 us
// streamed); up to one 128 x 128 tile a CU: those in the same way (512 rows of
// 5120 x 5120: 28.9 against 32.5 us); then two of these a CU, two blocks ahead
// (2048 rows of 2560 x 9728: 72.4 against 93.0 us).
// 256 x 256 tiles where they fill half of the CUs (2048 rows of 5120 x 5120: 70.3
// against 72.7 us, of 17408 x 5120: 190 against 242 us), 128 x 128 ones take more
// than one round (256 rows of 32768 x 5120: 93.0 against 73.9 us) and at most a
// quarter of what they cover is padding that smaller ones do not have (257 rows of
// 17408 x 5120: 69.5 against 46.7 us, 128 of 34816 x 5120 74.4 against 72.4, 60000
// of 64 x 5120 86 against 72; 513 rows of 17408 x 5120 on the other side: 71.4
// against 81.7 us).
// Up to 64 rows leave half of a taller tile empty: one 64 x 128 tile a CU, and past
// that two, two blocks ahead (40 rows of 34816 x 5120: 53.4 us, 54.5 in 128 x 128
// and 69 in 256 x 256 tiles; 64 of 151,936 x 5120: 165, 185 and 220 us); up to 32
// the stream kernel, which reads W once for them (32 of 34816 x 5120: 44.9 against
// 51.0 us).
// An fp32 result's products run at half the rate, which favours the stream kernel
// longer (512 rows of 2560 x 9728: 35.9 against 53.9 us; not with 33 to 64 rows, for
// which it reads W twice: 64 of 151,936 x 5120 356 against 196 us) and leaves 256 x
// 256 without registers.
template <typename TY>
hipError_t matmul(const Call<TY>& c) {
    auto tiles = [&](int64_t h, int64_t w) { return ((c.M + h - 1) / h) * ((c.N + w - 1) / w); };
    const int64_t cus = gqk_cu_count();
    if (tiles(64, 128) <= (sizeof(TY) == 4 ? 3 * cus / 4 : cus / 2)) {
        // rows of X and of W a workgroup: tall ones read either side less often, as long as 3 in 4 CUs have one
        if (c.M <= 16) return stream<1, 2, 8, false>(c, (c.M + 15) / 16);
        if (c.M <= 64) return stream<2, 2, 8, false>(c, (c.M + 31) / 32);
        if (tiles(48, 64) >= 3 * cus / 4) return stream<3, 4, 8, false>(c, (c.M + 47) / 48);
        return stream<3, 2, 8, false>(c, (c.M + 47) / 48);
    }
    if (c.M <= 32) return stream<2, 2, 8, false>(c, (c.M + 31) / 32);
    if (tiles(64, 128) <= cus && (sizeof(TY) == 2 || c.M <= 64)) return tile<64, 128, 2, 4, 4, false>(c);
    if (c.M <= 64) return tile<64, 128, 2, 4, 2, false>(c);
    if constexpr (sizeof(TY) == 2) {
        const int64_t small = tiles(128, 128), large = tiles(256, 256);
        if (small <= cus) return tile<128, 128, 4, 2, 4, false>(c);
        if (large >= cus / 2 && small > 2 * cus && 3 * large < small) return tile<256, 256, 4, 2, 2, true>(c);
    }
    return tile<128, 128, 4, 2, 2, false>(c);
}

// A launch has fewer than 2^23 workgroups of eight wavefronts, the last round's
// quarters among them: more rows than that many tiles of 128 x 128 have are
// multiplied by several.
template <typename TY>
hipError_t matmul_rows(Call<TY> c) {
    const int64_t M = c.M, most = ((1 << 23) - 1024) / ((c.N + 127) / 128) * 128;
    for (int64_t m = 0; m < M; m += most) {
        c.M = M - m < most ? M - m : most;
        const hipError_t e = matmul(c);
        if (e != hipSuccess) return e;
        c.X += most * c.ldx;
        c.xs += most;
        c.Y += most * c.ldy;
    }
    return hipSuccess;
}

// The slots of a tile, by those that an expert has on average (the experts'
// popularity as of normal logits); the table serves every product of a layer, so N,
// K and the type do not count.  us a call at 16, 64, 128 and 256 slots a tile, bf16:
//   64 experts        1408 x 2816              2816 x 704
//     8 slots each     45   43   44   73        27   28   33   35
//    24                66   48   57   77        39   33   34   41
//    48                92   67   61   81        59   40   38   55
//   128               215  107  113   96       123   54   47   71
//   320               480  192  179  151       278  107   74   84
//   400               587  230  197  186       375  149  111  154
//   750              1056  388  323  284       733  266  213  194
// The borders are compromises: 320 slots of long rows would take 256 to a tile, 400
// of short ones 128, and an fp32 result, whose tiles of 256 have 128 columns, 128
// throughout (64 experts of 1408 x 2816, 400 slots: 285 against 304 us).
int tile_rows(int64_t S, int n_experts) {
    const int64_t E = n_experts;
    return S <= 8 * E ? 16 : S <= 48 * E ? 64 : S <= 320 * E ? 128 : 256;
}

// Few slots an expert.  There are many workgroups, so wavefronts that share one
// cost more (the join, the blocks that do not divide) than they hide, but for
// long rows (8 tokens x 8 of 128 experts, 704 x 2816: 17.7, 17.7 and 20.7 us
// with 2, 4 and 8 wavefronts; 2816 x 704: 18.4, 21.9 and 31.6 us; 2 tokens x 4
// of 16, 2560 x 9728: 35.7, 28.4 and 29.6 us).
template <typename TY>
hipError_t stream_id(const Call<TY>& c, int64_t gm) {
    if (c.K <= 8 * BLK) return stream<1, 2, 2, true>(c, gm);
    if (c.K <= 32 * BLK) return stream<1, 2, 4, true>(c, gm);
    return stream<1, 2, 8, true>(c, gm);
}

// Many slots an expert: tiles of h = 128 or 256 slots.  Short rows take 0.6 to
// 0.92 of the tile kernels' time (500 tokens x 2 of 8 experts, 400 x 400: 11.2
// against 18.7 us; 3015 x 4 of 16, 2816 x 768: 59.9 against 68.6 us; 3015 x 2 of
// 4, 2100 x 256: 43.4 against 47.0 us).
hipError_t many_id(const Call<uint16_t>& c, int64_t gm, int h, int n_experts) {
    if (c.K > 0 && c.K <= 6 * BLK) {
        const int64_t n_tiles = (c.M + h - 1) / h + n_experts / 2;  // (an expert's last is half full)
        return h == 128 ? short_id<4>(c, gm, n_tiles) : short_id<8>(c, gm, n_tiles);
    }
    if (h == 128) return tile_id<128, 128, 2, 2, 2, false>(c, gm);
    return tile_id<256, 256, 4, 2, 2, false>(c, gm);
}
hipError_t many_id(const Call<float>& c, int64_t gm, int h, int) {
    if (h == 128) return tile_id<128, 128, 2, 2, 2, false>(c, gm);
    return tile_id<256, 128, 4, 2, 2, false>(c, gm);
}

// Rows of X that lie 2^31 bytes and more apart: the tile kernels again, with
// pointers.  Where there are few tiles, eight wavefronts and one tile of columns
// a workgroup take the shorter tiles too: 33 and 132 slots for each of 32 and 8
// experts of 768 x 2816, 32.8 and 35.3 us (two tiles a workgroup: 41.1 and 50.7
// us), fp32 46.1 and 49.9 (47.5 and 70); from 517 tiles on the other way round:
// 62 slots for each of 32 of 1408 x 2816 59.8 us (64.8), of 64 of 768 x 2816 62.6
// (69.7), fp32 80.0 (97.1), 31 for each of 256 of 1408 x 2816 247 us (360).
template <typename TY>
hipError_t far_id(const Call<TY>& c, int64_t gm, int h) {
    const bool few = 2 * gm * ((c.N + 127) / 128) <= 3 * (int64_t)gqk_cu_count();
    if (h == 64 && !few) return tile_id<64, 128, 1, 4, 2, true>(c, gm);
    if (h == 128 && !few) return tile_id<128, 128, 2, 2, 2, true>(c, gm);
    return tile_id<256, 128, 4, 2, 2, true>(c, gm);
}

template <typename TY>
hipError_t matmul_id(Call<TY> c, int n_experts, const int32_t* ids, int n_tokens, int top_k, int x_per_slot,
                     const float* route_w, int y_dtype, void* ws) {
    const int S = n_tokens * top_k;
    const WsLayout L = layout(n_experts, S, c.N, y_dtype, route_w != nullptr);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int* hdr = reinterpret_cast<int*>(base);
    auto* tiles = reinterpret_cast<TileEntry*>(base + L.off_tile);
    int* slot_e = reinterpret_cast<int*>(base + L.off_expert);
    int* slot = reinterpret_cast<int*>(base + L.off_slot);
    TY* y = c.Y;
    if (route_w) c.Y = reinterpret_cast<TY*>(base + L.off_out);
    c.M = S;
    c.ldy = c.N;
    const int h = L.TM, gm = L.max_tiles;
    const bool small = ids && S <= SMALL && h == 16;
    c.t = Table{hdr, tiles, slot_e, slot, n_experts, S, top_k, x_per_slot, small ? ids : nullptr, !route_w};
    const int64_t rows = x_per_slot ? S : n_tokens;
    // (one tile of columns a workgroup: more than 320 slots for each expert, so a Y of 600 GB; before anything is
    // launched)
    if (h == 256 && !grid_ok(gm * ((c.N + 127) / 128), 512)) return hipErrorInvalidValue;
    if (ids && !small) {
        hipLaunchKernelGGL((k_f8_plan<TY>), dim3(n_experts + 1), dim3(S <= 4096 ? 256 : 1024), 0, c.s, ids, S,
                           n_experts, h, hdr, tiles, slot_e, slot, route_w ? nullptr : y, c.N);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipError_t e;
    if (h == 16) e = stream_id(c, gm);
    else if (rows * c.ldx >= INT_MAX) e = far_id(c, gm, h);
    else if (h == 64) e = tile_id<64, 128, 1, 4, 2, false>(c, gm);
    else e = many_id(c, gm, h, n_experts);
    if (e != hipSuccess || !route_w) return e;
    constexpr int V = 16 / sizeof(TY);
    if (c.N % V == 0) return combine<V>(c.Y, slot_e, route_w, n_tokens, top_k, c.N, y, c.s);
    return combine<1>(c.Y, slot_e, route_w, n_tokens, top_k, c.N, y, c.s);
}

}  // namespace

hipError_t gqk_f8_matmul(const uint8_t* W, const float* ws, int64_t N, int64_t K, const uint8_t* X, const float* xs,
                         int64_t M, int64_t ldx, int64_t xs_ld, void* Y, int y_dtype, int64_t ldy, hipStream_t s) {
    if (y_dtype == gqd::DT_F32)
        return matmul_rows(Call<float>{W, ws, N, K, X, xs, M, ldx, xs_ld, static_cast<float*>(Y), ldy, Table{}, s});
    return matmul_rows(Call<uint16_t>{W, ws, N, K, X, xs, M, ldx, xs_ld, static_cast<uint16_t*>(Y), ldy, Table{}, s});
}

size_t gqk_f8_matmul_id_ws_bytes(int n_experts, int n_tokens, int top_k, int64_t N, int y_dtype, int weighted) {
    return layout(n_experts, (int64_t)n_tokens * top_k, N, y_dtype, weighted).total;
}

hipError_t gqk_f8_matmul_id(const uint8_t* W, const float* wsc, int n_experts, int64_t N, int64_t K,
                            const int32_t* ids, int n_tokens, int top_k, const uint8_t* X, const float* xs,
                            int64_t ldx, int64_t xs_ld, int x_per_slot, const float* route_w, void* Y, int y_dtype,
                            void* ws, hipStream_t s) {
    if (y_dtype == gqd::DT_F32)
        return matmul_id(Call<float>{W, wsc, N, K, X, xs, 0, ldx, xs_ld, static_cast<float*>(Y), 0, Table{}, s},
                         n_experts, ids, n_tokens, top_k, x_per_slot, route_w, y_dtype, ws);
    return matmul_id(Call<uint16_t>{W, wsc, N, K, X, xs, 0, ldx, xs_ld, static_cast<uint16_t*>(Y), 0, Table{}, s},
                     n_experts, ids, n_tokens, top_k, x_per_slot, route_w, y_dtype, ws);
}

hipError_t gqk_f8_matmul_id_bad_count(const void* ws, hipStream_t s, int32_t* n_bad) {
    hipError_t e = hipMemcpyAsync(n_bad, ws, sizeof(int32_t), hipMemcpyDeviceToHost, s);
    if (e != hipSuccess) return e;
    return hipStreamSynchronize(s);
}
