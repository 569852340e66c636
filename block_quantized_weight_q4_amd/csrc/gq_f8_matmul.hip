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
#include <stdint.h>

#include "gq_f8_device.h"
#include "gq_f8_internal.h"
#include "gq_f8_stream.h"

using namespace gqf8;

namespace {

// ------------------------------------------------- slots by expert (plan) ----
// Workspace: header (int [0] = invalid ids), the first slot and the first tile
// of each expert (n_experts + 1 entries, the last one the totals), each slot's
// expert (-1: invalid id), the slots by expert, the per-slot outputs of a
// weighted product.
struct WsLayout {
    size_t off_first, off_tile, off_expert, off_slot, off_out, total;
};

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

WsLayout layout(int n_experts, int64_t S, int64_t N, int y_dtype, int weighted) {
    WsLayout L;
    L.off_first = 256;
    L.off_tile = L.off_first + up256(4 * ((size_t)n_experts + 1));
    L.off_expert = L.off_tile + up256(4 * ((size_t)n_experts + 1));
    L.off_slot = L.off_expert + up256(4 * (size_t)S);
    L.off_out = L.off_slot + up256(4 * (size_t)S);
    L.total = L.off_out + (weighted ? (size_t)S * (size_t)N * (y_dtype == gqd::DT_F32 ? 4 : 2) : 0);
    return L;
}

struct Table {
    const int *first, *tile, *slot;
    int n_experts, S, top_k, per_slot;
};

constexpr int PLAN_THREADS = 256;
constexpr int MAX_E = 4096;

// Workgroup e < n_experts lists the slots of expert e (their order among
// themselves does not reach any result: each output row is computed on its
// own).  The last workgroup counts the slots of every expert and writes the
// first slot, the first tile (of TM slots) and the totals, and zeroes the
// output rows of invalid slots.
template <typename TY>
__global__ __launch_bounds__(PLAN_THREADS) void k_f8_plan(const int32_t* __restrict__ ids, int S, int n_experts,
                                                          int TM, int* __restrict__ hdr, int* __restrict__ first,
                                                          int* __restrict__ tile, int* __restrict__ slot_e,
                                                          int* __restrict__ slot, TY* __restrict__ y, int64_t N) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int e = blockIdx.x;
    if (e < n_experts) {
        __shared__ int n_less, n_here;
        if (tid == 0) {
            n_less = 0;
            n_here = 0;
        }
        __syncthreads();
        int less = 0;
        for (int s = tid; s < S; s += PLAN_THREADS) less += ids[s] >= 0 && ids[s] < e;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) less += __shfl_xor(less, off, 64);
        if (lane == 0) atomicAdd(&n_less, less);
        __syncthreads();
        const int base = n_less;
        for (int s0 = 0; s0 < S; s0 += PLAN_THREADS) {
            const int s = s0 + tid;
            const bool mine = s < S && ids[s] == e;
            const uint64_t vote = __ballot(mine);
            if (vote == 0) continue;
            int at = 0;
            if (lane == 0) at = atomicAdd(&n_here, __popcll(vote));
            at = __builtin_amdgcn_readfirstlane(at);
            if (mine) slot[base + at + __popcll(vote & ((1ull << lane) - 1))] = s;
        }
        return;
    }
    __shared__ int count[MAX_E];
    __shared__ int n_bad;
    if (tid == 0) n_bad = 0;
    for (int i = tid; i < n_experts; i += PLAN_THREADS) count[i] = 0;
    __syncthreads();
    for (int s = tid; s < S; s += PLAN_THREADS) {
        const int i = ids[s];
        const bool ok = i >= 0 && i < n_experts;
        slot_e[s] = ok ? i : -1;
        atomicAdd(ok ? &count[i] : &n_bad, 1);
    }
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
            first[i] = ra;
            tile[i] = rb;
            ra += count[i];
            rb += (count[i] + TM - 1) / TM;
        }
        if (tid == 63) {
            first[n_experts] = ia;
            tile[n_experts] = ib;
            hdr[0] = n_bad;
        }
    }
    if (y && n_bad)
        for (int s = 0; s < S; ++s) {
            const int i = ids[s];
            if (i < 0 || i >= n_experts)
                for (int64_t n = tid; n < N; n += PLAN_THREADS) store_as(y + s * N + n, 0.0f);
        }
}

// The expert and the slots [start, start + rows) of tile i; rows == 0 where
// the table has no such tile.  Every field is clamped to its range.
__device__ __forceinline__ void tile_of(const Table& t, int i, int TM, int& e, int& start, int& rows) {
    int lo = 0, hi = t.n_experts;  // the last e with tile[e] <= i
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.tile[mid] <= i) lo = mid;
        else hi = mid;
    }
    e = lo;
    rows = 0;
    start = 0;
    if (i >= t.tile[t.n_experts]) return;
    const int64_t a = (int64_t)t.first[e] + ((int64_t)i - t.tile[e]) * TM;
    int64_t b = t.first[e + 1];
    b = b < t.S ? b : t.S;
    if (a < 0 || a >= b) return;
    start = (int)a;
    rows = (int)(b - a < TM ? b - a : TM);
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
// Both tiles of a 128-input block go to LDS by global-to-LDS copies, NB - 1
// blocks ahead, in rows of 128 bytes whose 16-byte chunks are swizzled so that
// operand reads cover all banks; the block's activation scales come along.
// One barrier a block.
template <int BM, int BN, int WM, int WN, int NB, typename TY, bool ROUTED>
struct Tile {
    static constexpr int WV = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
    static constexpr int XI = BM / 8 / WV, WI = BN / 8 / WV;  // copies of a wavefront and block
    static constexpr int SX = (BM + BN) * BLK, STAGE = SX + WV * 256;
    static constexpr int LOADS = XI + WI + 1;
    static_assert(BM % (8 * WV) == 0 && BN % (8 * WV) == 0 && WV > BM / 64 && BN / WN <= BLK, "tile shape");

    static __device__ __forceinline__ void run(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                               int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                               const float* __restrict__ xs, int64_t ldx, int64_t xs_ld,
                                               TY* __restrict__ Y, int64_t ldy, int64_t m0, int64_t n0, int rows,
                                               int start, const Table& t, uint8_t* smem) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int fr = lane & 15, fq = lane >> 4;
        const int wm = (wave % WM) * (BM / WM), wn = (wave / WM) * (BN / WN);
        const int KB = (int)((K + BLK - 1) / BLK);
        const int64_t w_rows = N - n0 < BN ? N - n0 : BN;
        const Rsrc wr = make_rsrc(W + n0 * K, w_rows * K);
        const Rsrc xr = make_rsrc(X + m0 * ldx, (int64_t)rows * ldx);  // (dense)
        auto slot_of = [&](int i) -> int64_t {
            const unsigned s = (unsigned)t.slot[start + (i < rows ? i : rows - 1)];
            return s < (unsigned)t.S ? (int64_t)s : t.S - 1;
        };
        auto x_row = [&](int i) -> int64_t {
            if constexpr (ROUTED) return t.per_slot ? slot_of(i) : slot_of(i) / t.top_k;
            else return m0 + (i < rows ? i : rows - 1);
        };
        // copies: wavefront w brings rows 8 (w + WV u) .. + 7 of either tile
        uint32_t xoff[XI], woff[WI];
        const uint8_t* xp[XI];
#pragma unroll
        for (int u = 0; u < XI; ++u) {
            const int r = 8 * (wave + WV * u) + (lane >> 3);
            if constexpr (ROUTED) xp[u] = X + x_row(r) * ldx;
            else xoff[u] = (uint32_t)(r * ldx);
        }
#pragma unroll
        for (int u = 0; u < WI; ++u) woff[u] = (uint32_t)((8 * (wave + WV * u) + (lane >> 3)) * K);
        // the chunk of row r that its lane copies: (lane % 8) ^ (r / 2 % 8), r = 8 (wave + WV u) + lane / 8
        const uint32_t chunk = 16u * (uint32_t)((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
        static_assert(WV % 2 == 0, "the swizzle of a lane's rows is the same for all of its copies");
        // one copy of 64 scales: wavefronts below BM / 64 those of X, the others W's (of wavefront w's columns: lane w)
        const float* sp;
        int64_t sstep;
        if (wave < BM / 64) {
            sp = xs + x_row(64 * wave + lane);
            sstep = xs_ld;
        } else {
            const int64_t n = n0 + (lane % WV / WM) * (BN / WN);
            sp = wsc + ((n < N ? n : N - 1) / BLK) * KB;
            sstep = 1;
        }
        auto load = [&](int kb) {
            uint8_t* d = smem + (kb % NB) * STAGE;
            const int64_t k = (int64_t)kb * BLK + chunk;
            const bool in = k < K;
#pragma unroll
            for (int u = 0; u < XI; ++u) {
                uint8_t* l = d + (wave + WV * u) * 1024;
                if constexpr (ROUTED) copy16(xp[u] + (in ? k : 0), l);
                else copy16(xr, in ? xoff[u] + (uint32_t)k : NOWHERE, l);
            }
#pragma unroll
            for (int u = 0; u < WI; ++u)
                copy16(wr, in ? woff[u] + (uint32_t)k : NOWHERE, d + BM * BLK + (wave + WV * u) * 1024);
            copy4(sp + (kb < KB ? kb : KB - 1) * sstep, d + SX + wave * 256);
        };
        f32x4 acc[NT][MT];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{};
        if (KB > 0) {
#pragma unroll
            for (int s = 0; s < NB - 1; ++s) load(s);
            wait_copies<(NB - 2) * LOADS>();
            gqd::lds_barrier();
        }
        // 16-byte positions of this lane's two chunks of an operand row (rows 16 i + fr: the same for every i)
        const int p0 = pos128(fr, fq), p1 = pos128(fr, 4 + fq);
        for (int kb = 0; kb < KB; ++kb) {
            load(kb + NB - 1);
            const uint8_t* d = smem + (kb % NB) * STAGE;
            const u32x4* dx = reinterpret_cast<const u32x4*>(d + wm * BLK);
            const u32x4* dw = reinterpret_cast<const u32x4*>(d + (BM + wn) * BLK);
            const float* ds = reinterpret_cast<const float*>(d + SX);
            const float s_w = ds[(BM / 64) * 64 + wave];
            float s[MT];
            i32x8 x[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                x[j] = join(dx[128 * j + p0], dx[128 * j + p1]);
                s[j] = s_w * ds[wm + 16 * j + fr];
            }
            if constexpr (sizeof(TY) == 4) {
                Wide xw[MT];
#pragma unroll
                for (int j = 0; j < MT; ++j) xw[j] = widen(x[j]);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const Wide a = widen(join(dw[128 * i + p0], dw[128 * i + p1]));
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        const f32x4 p = mfma16(a, xw[j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s[j], acc[i][j][r]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const i32x8 a = join(dw[128 * i + p0], dw[128 * i + p1]);
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        const f32x4 p = mfma8(a, x[j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s[j], acc[i][j][r]);
                    }
                }
            }
            wait_copies<(NB - 2) * LOADS>();
            gqd::lds_barrier();
        }
        wait_copies<0>();
        const bool vec = (ldy & 3) == 0;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row = wm + 16 * j + fr;
            if (row >= rows) continue;
            TY* y = Y + (ROUTED ? slot_of(row) : m0 + row) * ldy;
#pragma unroll
            for (int i = 0; i < NT; ++i) store4(y, n0 + wn + 16 * i + 4 * fq, N, vec, acc[i][j]);
        }
    }
};

template <int BM, int BN, int WM, int WN, int NB, typename TY, bool ROUTED>
__global__ __launch_bounds__(64 * WM * WN) void k_f8_tile(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                                          int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                                          const float* __restrict__ xs, int64_t M, int64_t ldx,
                                                          int64_t xs_ld, TY* __restrict__ Y, int64_t ldy, int gm,
                                                          int gn, Table t) {
    using T = Tile<BM, BN, WM, WN, NB, TY, ROUTED>;
    __shared__ __align__(16) uint8_t smem[NB * T::STAGE];
    const int id = xcd_order(blockIdx.x, gm * gn);
    int tm, tn, e = 0, start = 0, rows;
    if constexpr (ROUTED) {
        tm = id / gn;  // an expert's tiles side by side: they share its rows of X
        tn = id % gn;
        tile_of(t, tm, BM, e, start, rows);
        if (rows == 0) return;
        W += (int64_t)e * N * K;
        wsc += (int64_t)e * ((N + BLK - 1) / BLK) * ((K + BLK - 1) / BLK);
    } else {
        // bands of at most 12 row tiles
        const int bands = (gm + 11) / 12, h = (gm + bands - 1) / bands;
        const int band = id / (h * gn), hb = gm - band * h < h ? gm - band * h : h;
        const int r = id - band * h * gn;
        tm = band * h + r % hb;
        tn = r / hb;
        const int64_t left = M - (int64_t)tm * BM;
        rows = (int)(left < BM ? left : BM);
    }
    T::run(W, wsc, N, K, X, xs, ldx, xs_ld, Y, ldy, (int64_t)tm * BM, (int64_t)tn * BN, rows, start, t, smem);
}

// A few rows: the stream kernel, 16 MT rows of X and 16 NT of W a workgroup.
template <int MT, int NT, int WV, int D, typename TY, bool ROUTED>
__global__ __launch_bounds__(64 * WV) void k_f8_stream(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                                       int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                                       const float* __restrict__ xs, int64_t M, int64_t ldx,
                                                       int64_t xs_ld, TY* __restrict__ Y, int64_t ldy, int gn,
                                                       Table t) {
    constexpr int RING = WV * D * Stream<MT, NT, X_E4M3, 16 * MT>::BYTES, JOIN = WV * NT * MT * 1024;
    __shared__ __align__(16) uint8_t smem[RING > JOIN ? RING : JOIN];
    const int tn = blockIdx.x % gn, tm = blockIdx.x / gn;
    int e = 0, start = 0, rows;
    if constexpr (ROUTED) {
        tile_of(t, tm, 16 * MT, e, start, rows);
        if (rows == 0) return;
        W += (int64_t)e * N * K;
        wsc += (int64_t)e * ((N + BLK - 1) / BLK) * ((K + BLK - 1) / BLK);
    } else {
        const int64_t left = M - (int64_t)tm * (16 * MT);
        rows = (int)(left < 16 * MT ? left : 16 * MT);
    }
    auto row_of = [&](int i) -> int64_t {
        const int c = i < rows ? i : rows - 1;
        if constexpr (ROUTED) {
            const unsigned s = (unsigned)t.slot[start + c];
            return s < (unsigned)t.S ? (int64_t)s : t.S - 1;
        } else {
            return (int64_t)tm * (16 * MT) + c;
        }
    };
    stream_tile<MT, NT, WV, D, X_E4M3, 16 * MT, TY>(
        W, wsc, (int64_t)tn * (16 * NT), N, K, X, xs, ldx, xs_ld, rows, (ldy & 3) == 0,
        [&](int i) { return ROUTED && !t.per_slot ? row_of(i) / t.top_k : row_of(i); },
        [&](int i) { return Y + row_of(i) * ldy; }, smem);
}

// y[t][n] = sum_j rw[t][j] slot[t][j][n], j in increasing order, slots of
// invalid ids left out.
template <typename TY>
__global__ __launch_bounds__(256) void k_f8_combine(const TY* __restrict__ slots, const int* __restrict__ slot_e,
                                                    const float* __restrict__ rw, int n_tokens, int top_k, int64_t N,
                                                    TY* __restrict__ y) {
    const int64_t total = (int64_t)n_tokens * N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / N, n = i - t * N;
        float sum = 0.0f;
        for (int j = 0; j < top_k; ++j) {
            const int64_t s = t * top_k + j;
            if (slot_e[s] < 0) continue;
            float v;
            if constexpr (sizeof(TY) == 4) v = slots[s * N + n];
            else v = gqd::bf2f(slots[s * N + n]);
            sum = __builtin_fmaf(rw[s], v, sum);
        }
        store_as(y + i, sum);
    }
}

bool grid_ok(int64_t groups, int threads) { return groups * threads < ((int64_t)1 << 32); }

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
template <int MT, int NT, int WV, int D, bool ROUTED, typename TY>
hipError_t stream(const Call<TY>& c, int64_t gm) {
    const int64_t gn = (c.N + 16 * NT - 1) / (16 * NT);
    if (!grid_ok(gn * gm, 64 * WV)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_f8_stream<MT, NT, WV, D, TY, ROUTED>), dim3((unsigned)(gn * gm)), dim3(64 * WV), 0, c.s, c.W,
                       c.wsc, c.N, c.K, c.X, c.xs, c.M, c.ldx, c.xs_ld, c.Y, c.ldy, (int)gn, c.t);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NB, bool ROUTED, typename TY>
hipError_t tile(const Call<TY>& c, int64_t gm) {
    const int64_t gn = (c.N + BN - 1) / BN;
    if (!grid_ok(gn * gm, 64 * WM * WN)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_f8_tile<BM, BN, WM, WN, NB, TY, ROUTED>), dim3((unsigned)(gn * gm)), dim3(64 * WM * WN), 0,
                       c.s, c.W, c.wsc, c.N, c.K, c.X, c.xs, c.M, c.ldx, c.xs_ld, c.Y, c.ldy, (int)gm, (int)gn, c.t);
    return hipGetLastError();
}

template <typename TY>
hipError_t matmul(const Call<TY>& c) {
    auto tiles = [&](int h) { return (c.M + h - 1) / h; };
    if (c.M <= 16) return stream<1, 2, 8, 1, false>(c, tiles(16));
    if (c.M <= 256) return stream<2, 2, 8, 1, false>(c, tiles(32));
    if constexpr (sizeof(TY) == 2)
        if (c.M >= 1024 && c.N >= 2048) return tile<256, 256, 4, 2, 2, false>(c, tiles(256));
    return tile<128, 128, 2, 2, 2, false>(c, tiles(128));
}

// Rows of a tile of slots, from what every product of a layer has in common.
int tile_rows(int64_t S, int n_experts) {
    return S <= 16 * (int64_t)n_experts ? 16 : S <= 64 * (int64_t)n_experts ? 32 : 128;
}

template <typename TY>
hipError_t matmul_id(Call<TY> c, int n_experts, const int32_t* ids, int n_tokens, int top_k, int x_per_slot,
                     const float* route_w, int y_dtype, void* ws) {
    const int S = n_tokens * top_k;
    const WsLayout L = layout(n_experts, S, c.N, y_dtype, route_w != nullptr);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int* hdr = reinterpret_cast<int*>(base);
    int* first = reinterpret_cast<int*>(base + L.off_first);
    int* tile_at = reinterpret_cast<int*>(base + L.off_tile);
    int* slot_e = reinterpret_cast<int*>(base + L.off_expert);
    int* slot = reinterpret_cast<int*>(base + L.off_slot);
    TY* y = c.Y;
    if (route_w) c.Y = reinterpret_cast<TY*>(base + L.off_out);
    c.M = S;
    c.ldy = c.N;
    c.t = Table{first, tile_at, slot, n_experts, S, top_k, x_per_slot};
    const int h = tile_rows(S, n_experts);
    if (ids) {
        hipLaunchKernelGGL((k_f8_plan<TY>), dim3(n_experts + 1), dim3(PLAN_THREADS), 0, c.s, ids, S, n_experts, h, hdr,
                           first, tile_at, slot_e, slot, route_w ? nullptr : y, c.N);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // tiles of the worst case: every expert may end with a partial one
    const int64_t gm = S / h + (S < n_experts ? S : n_experts);
    hipError_t e;
    if (h == 16) e = stream<1, 2, 8, 1, true>(c, gm);
    else if (h == 32) e = stream<2, 2, 8, 1, true>(c, gm);
    else e = tile<128, 128, 2, 2, 2, true>(c, gm);
    if (e != hipSuccess || !route_w) return e;
    const int64_t want = ((int64_t)n_tokens * c.N + 255) / 256;
    hipLaunchKernelGGL((k_f8_combine<TY>), dim3((unsigned)(want < 65536 ? want : 65536)), dim3(256), 0, c.s, c.Y,
                       slot_e, route_w, n_tokens, top_k, c.N, y);
    return hipGetLastError();
}

}  // namespace

hipError_t gqk_f8_matmul(const uint8_t* W, const float* ws, int64_t N, int64_t K, const uint8_t* X, const float* xs,
                         int64_t M, int64_t ldx, int64_t xs_ld, void* Y, int y_dtype, int64_t ldy, hipStream_t s) {
    if (y_dtype == gqd::DT_F32)
        return matmul(Call<float>{W, ws, N, K, X, xs, M, ldx, xs_ld, static_cast<float*>(Y), ldy, Table{}, s});
    return matmul(Call<uint16_t>{W, ws, N, K, X, xs, M, ldx, xs_ld, static_cast<uint16_t*>(Y), ldy, Table{}, s});
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
