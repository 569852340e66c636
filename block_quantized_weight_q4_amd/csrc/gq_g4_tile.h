// gq_g4_tile.h -- which rows of X a workgroup of a product of many rows works on
// (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_g4_device.h"
#include "gq_g4_internal.h"

namespace gqg4 {

// Workgroups go to the 8 XCDs in turn, so XCD x takes a run of neighbouring tiles
// (each XCD has an L2 of its own).
__device__ __forceinline__ int xcd_order(int id, int total) {
    const int x = id & 7, q = total >> 3, r = total & 7;
    return x * q + (x < r ? x : r) + (id >> 3);
}

// The rows of one tile: [row0, row0 + rows) of X, of expert e.
struct RowTile {
    int e, rows;
    int64_t row0;
};

// Rows of expert i, [begin, begin + count): offsets clamped to 0..M.
__device__ __forceinline__ int rows_of(const int32_t* __restrict__ offsets, int64_t M, int i, int64_t& begin) {
    int64_t a = offsets[i], b = offsets[i + 1];
    a = a < 0 ? 0 : a > M ? M : a;
    b = b < 0 ? 0 : b > M ? M : b;
    begin = a;
    return b > a ? (int)(b - a) : 0;
}

// Every expert's rows are cut into tiles of at most TM; total_tiles counts them.
// Every wavefront counts for itself, a lane a run of the experts; `pick` is called
// with the total and gives the number of the wavefront's own tile, or -1.  False
// where there is none.
template <typename Pick>
__device__ __forceinline__ bool tile_of(const int32_t* __restrict__ offsets, int E, int64_t M, int TM, Pick pick,
                                        RowTile& t) {
    const int lane = threadIdx.x & 63;
    const int per = (E + 63) / 64;
    const int lo = lane * per < E ? lane * per : E, hi = lo + per < E ? lo + per : E;
    int64_t begin;
    int n = 0;
    for (int i = lo; i < hi; ++i) n += (rows_of(offsets, M, i, begin) + TM - 1) / TM;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(incl, off, 64);
        if (lane >= off) incl += v;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63);
    const int want = pick(total);
    if (want < 0 || want >= total) return false;
    const uint64_t hit = __ballot(incl > want);  // (not empty: the last lane's is the total)
    const int l = __builtin_ctzll(hit);
    int left = want - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l));
    for (int i = l * per; i < E; ++i) {
        const int rows = rows_of(offsets, M, i, begin), tiles = (rows + TM - 1) / TM;
        if (left >= 0 && left < tiles) {
            t.e = i;
            t.row0 = begin + (int64_t)left * TM;
            t.rows = rows - left * TM < TM ? rows - left * TM : TM;
            return true;
        }
        left -= tiles;
    }
    return false;
}

// Weights of expert e.
__device__ __forceinline__ G4Weights of_expert(G4Weights w, int e) {
    const int64_t KG = (w.K + w.group - 1) / w.group;
    w.W += (int64_t)e * w.N * (w.K / 2);
    w.scales += (int64_t)e * w.N * KG;
    if (w.zeros) w.zeros += (int64_t)e * w.N * KG;
    return w;
}

// Workgroups of one launch (of at most 256 threads; a launch has fewer than 2^32).
constexpr int64_t MOST_GROUPS = (int64_t)1 << 23;

// Most tiles there can be: every expert ends with a partial one.
inline int64_t most_tiles(int64_t M, int E, int TM) { return M / TM + (M < E ? M : E); }

}  // namespace gqg4
