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

// ------------------------------------------------------------- the product ----
constexpr int TM = 64, TN = 64;

// One 64 x 64 tile of Y: 4 wavefronts, each 32 x 32 as 2 x 2 MFMA tiles.
template <typename TY, bool ROUTED>
__global__ __launch_bounds__(256) void k_f8_matmul(const uint8_t* __restrict__ W, const float* __restrict__ wsc,
                                                   int64_t N, int64_t K, const uint8_t* __restrict__ X,
                                                   const float* __restrict__ xs, int64_t M, int64_t ldx,
                                                   int64_t xs_ld, TY* __restrict__ Y, int64_t ldy, int gn, Table t) {
    __shared__ __align__(16) uint8_t lx[TM * BLK], lw[TN * BLK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tn = blockIdx.x % gn, tm = blockIdx.x / gn;
    const int64_t n0 = (int64_t)tn * TN;
    const int64_t KB = (K + BLK - 1) / BLK;
    int e = 0, start = 0, rows;
    if constexpr (ROUTED) {
        tile_of(t, tm, TM, e, start, rows);
        if (rows == 0) return;
        W += (int64_t)e * N * K;
        wsc += (int64_t)e * ((N + BLK - 1) / BLK) * KB;
    } else {
        const int64_t left = M - (int64_t)tm * TM;
        rows = (int)(left < TM ? left : TM);
    }
    // rows of X and of Y that tile row i stands for
    auto y_row = [&](int i) -> int64_t {
        if constexpr (ROUTED) {
            const unsigned s = (unsigned)t.slot[start + (i < rows ? i : 0)];
            return s < (unsigned)t.S ? (int64_t)s : t.S - 1;
        } else {
            return (int64_t)tm * TM + (i < rows ? i : 0);
        }
    };
    auto x_row = [&](int i) -> int64_t {
        const int64_t r = y_row(i);
        return ROUTED && !t.per_slot ? r / t.top_k : r;
    };
    const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
    const int fr = lane & 15, fq = lane >> 4;
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{};
    int64_t xr[2];  // rows of X whose scales this lane uses
#pragma unroll
    for (int j = 0; j < 2; ++j) xr[j] = x_row(wm + 16 * j + fr);
    int64_t lr[2];  // rows of X that this thread loads
#pragma unroll
    for (int i = 0; i < 2; ++i) lr[i] = x_row((tid + 256 * i) >> 3);

    for (int64_t b = 0; b < KB; ++b) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = tid + 256 * i, r = c >> 3, ch = c & 7;
            const int64_t k = b * BLK + 16 * ch;
            u32x4 vx{}, vw{};
            if (k < K && r < rows) vx = *reinterpret_cast<const u32x4*>(X + lr[i] * ldx + k);
            if (k < K && n0 + r < N) vw = *reinterpret_cast<const u32x4*>(W + (n0 + r) * K + k);
            const int at = r * BLK + ((ch ^ (r & 7)) << 4);  // swizzled: conflict-free reads
            *reinterpret_cast<u32x4*>(lx + at) = vx;
            *reinterpret_cast<u32x4*>(lw + at) = vw;
        }
        __syncthreads();
        i32x8 a[2], x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rw = wn + 16 * i + fr, rx = wm + 16 * i + fr;
            const int c0 = ((2 * fq) ^ (fr & 7)) << 4, c1 = ((2 * fq + 1) ^ (fr & 7)) << 4;
            a[i] = join(*reinterpret_cast<const u32x4*>(lw + rw * BLK + c0),
                        *reinterpret_cast<const u32x4*>(lw + rw * BLK + c1));
            x[i] = join(*reinterpret_cast<const u32x4*>(lx + rx * BLK + c0),
                        *reinterpret_cast<const u32x4*>(lx + rx * BLK + c1));
        }
        const float w_s = wsc[(n0 / BLK) * KB + b];  // (a 64-row tile lies in one block of 128 rows)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float s = w_s * xs[b * xs_ld + xr[j]];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x4 p;
                if constexpr (sizeof(TY) == 4) p = mfma16(widen(a[i]), widen(x[j]));
                else p = mfma8(a[i], x[j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s, acc[i][j][r]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = wm + 16 * j + fr;
        if (row >= rows) continue;
        TY* y = Y + y_row(row) * ldy;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t n = n0 + wn + 16 * i + 4 * fq + r;
                if (n < N) store_as(y + n, acc[i][j][r]);
            }
    }
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

template <typename TY>
hipError_t matmul(const uint8_t* W, const float* ws, int64_t N, int64_t K, const uint8_t* X, const float* xs,
                  int64_t M, int64_t ldx, int64_t xs_ld, TY* Y, int64_t ldy, hipStream_t s) {
    const int64_t gn = (N + TN - 1) / TN, gm = (M + TM - 1) / TM;
    if (!grid_ok(gn * gm, 256)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_f8_matmul<TY, false>), dim3((unsigned)(gn * gm)), dim3(256), 0, s, W, ws, N, K, X, xs, M,
                       ldx, xs_ld, Y, ldy, (int)gn, Table{});
    return hipGetLastError();
}

template <typename TY>
hipError_t matmul_id(const uint8_t* W, const float* wsc, int n_experts, int64_t N, int64_t K, const int32_t* ids,
                     int n_tokens, int top_k, const uint8_t* X, const float* xs, int64_t ldx, int64_t xs_ld,
                     int x_per_slot, const float* route_w, TY* Y, int y_dtype, void* ws, hipStream_t s) {
    const int S = n_tokens * top_k;
    const WsLayout L = layout(n_experts, S, N, y_dtype, route_w != nullptr);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int* hdr = reinterpret_cast<int*>(base);
    int* first = reinterpret_cast<int*>(base + L.off_first);
    int* tile = reinterpret_cast<int*>(base + L.off_tile);
    int* slot_e = reinterpret_cast<int*>(base + L.off_expert);
    int* slot = reinterpret_cast<int*>(base + L.off_slot);
    TY* out = route_w ? reinterpret_cast<TY*>(base + L.off_out) : Y;
    // tiles of the worst case: every expert may end with a partial one
    const int64_t gm = S / TM + (S < n_experts ? S : n_experts), gn = (N + TN - 1) / TN;
    if (!grid_ok(gm * gn, 256)) return hipErrorInvalidValue;
    if (ids) {
        hipLaunchKernelGGL((k_f8_plan<TY>), dim3(n_experts + 1), dim3(PLAN_THREADS), 0, s, ids, S, n_experts, TM, hdr,
                           first, tile, slot_e, slot, route_w ? nullptr : Y, N);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const Table t{first, tile, slot, n_experts, S, top_k, x_per_slot};
    hipLaunchKernelGGL((k_f8_matmul<TY, true>), dim3((unsigned)(gn * gm)), dim3(256), 0, s, W, wsc, N, K, X, xs,
                       (int64_t)0, ldx, xs_ld, out, N, (int)gn, t);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !route_w) return e;
    const int64_t want = ((int64_t)n_tokens * N + 255) / 256;
    hipLaunchKernelGGL((k_f8_combine<TY>), dim3((unsigned)(want < 65536 ? want : 65536)), dim3(256), 0, s, out,
                       slot_e, route_w, n_tokens, top_k, N, Y);
    return hipGetLastError();
}

}  // namespace

hipError_t gqk_f8_matmul(const uint8_t* W, const float* ws, int64_t N, int64_t K, const uint8_t* X, const float* xs,
                         int64_t M, int64_t ldx, int64_t xs_ld, void* Y, int y_dtype, int64_t ldy, hipStream_t s) {
    if (y_dtype == gqd::DT_F32)
        return matmul(W, ws, N, K, X, xs, M, ldx, xs_ld, static_cast<float*>(Y), ldy, s);
    return matmul(W, ws, N, K, X, xs, M, ldx, xs_ld, static_cast<uint16_t*>(Y), ldy, s);
}

size_t gqk_f8_matmul_id_ws_bytes(int n_experts, int n_tokens, int top_k, int64_t N, int y_dtype, int weighted) {
    return layout(n_experts, (int64_t)n_tokens * top_k, N, y_dtype, weighted).total;
}

hipError_t gqk_f8_matmul_id(const uint8_t* W, const float* wsc, int n_experts, int64_t N, int64_t K,
                            const int32_t* ids, int n_tokens, int top_k, const uint8_t* X, const float* xs,
                            int64_t ldx, int64_t xs_ld, int x_per_slot, const float* route_w, void* Y, int y_dtype,
                            void* ws, hipStream_t s) {
    if (y_dtype == gqd::DT_F32)
        return matmul_id(W, wsc, n_experts, N, K, ids, n_tokens, top_k, X, xs, ldx, xs_ld, x_per_slot, route_w,
                         static_cast<float*>(Y), y_dtype, ws, s);
    return matmul_id(W, wsc, n_experts, N, K, ids, n_tokens, top_k, X, xs, ldx, xs_ld, x_per_slot, route_w,
                     static_cast<uint16_t*>(Y), y_dtype, ws, s);
}

hipError_t gqk_f8_matmul_id_bad_count(const void* ws, hipStream_t s, int32_t* n_bad) {
    hipError_t e = hipMemcpyAsync(n_bad, ws, sizeof(int32_t), hipMemcpyDeviceToHost, s);
    if (e != hipSuccess) return e;
    return hipStreamSynchronize(s);
}
