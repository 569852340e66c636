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
#include "gq_g4_internal.h"
#include "gq_g4_tile.h"

using namespace gqg4;

namespace {

constexpr int BK = 64;     // rows of W (columns of dY) of a stage
constexpr int BN = 256;    // columns of a tile: 64 of each of the four wavefronts
constexpr int STAGES = 3;  // in LDS

struct Rows {
    const uint16_t* dY;
    int64_t M, lddy;
    uint16_t* dX;
    int64_t lddx;
    int n_experts;
    const int32_t* offsets;
};

// BM = 16 MT rows by BN columns.  DMA: rows of dY are whole 16-byte pieces, copied
// straight to LDS; otherwise they go through registers, element by element at
// their end.
template <typename T, int MT, bool DMA>
struct Tile {
    static constexpr int BM = 16 * MT;
    static constexpr int XB = BM * 128, WB = BK * (BN / 2), STAGE = XB + WB;
    static constexpr int XI = BM / 32, WI = 2;
    // scales of a wavefront's 64 columns (two groups at most) and a stage's 64 rows, two stages
    static constexpr int SCALES = 2 * 2 * BK * 8;
    static constexpr int BYTES = STAGES * STAGE + 4 * SCALES;

    static __device__ __forceinline__ void run(const G4Weights& wt, const uint16_t* __restrict__ dy, int64_t lddy,
                                               int rows, uint16_t* __restrict__ dx, int64_t lddx, int64_t k0,
                                               uint8_t* smem) {
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int fr = lane & 15, fq = lane >> 4;
        const int64_t N = wt.N, K = wt.K, row_bytes = K / 2, KG = (K + wt.group - 1) / wt.group;
        const int S = (int)((N + BK - 1) / BK);

        // dY: rows of 128 bytes, chunks swizzled by row pairs; wavefront w has rows 8 (w + 4 u) .. + 7
        const int xlr = 8 * wave + (lane >> 3), xchunk = 8 * ((lane & 7) ^ ((xlr >> 1) & 7));  // (elements)
        const uint16_t* xp[XI];
#pragma unroll
        for (int u = 0; u < XI; ++u) {
            const int r = xlr + 32 * u;
            xp[u] = dy + (int64_t)(r < rows ? r : rows - 1) * lddy;
        }
        // W: rows of 128 bytes; the 32-byte pieces of rows 8 apart are exchanged, so
        // that the four rows that the lanes read at once are in different banks
        auto load = [&](int s) {
            uint8_t* d = smem + (s % STAGES) * STAGE;
            const int64_t n = (int64_t)s * BK;
            const int left = n < N ? (int)(N - n < BK ? N - n : BK) : 0;
#pragma unroll
            for (int u = 0; u < XI; ++u) {
                uint8_t* l = d + (wave + 4 * u) * 1024;
                if constexpr (DMA) {
                    // (past the row's end its first piece, which meets weights of zero)
                    copy16(reinterpret_cast<const uint8_t*>(xp[u] + (xchunk < left ? n + xchunk : 0)), l);
                } else {
                    u32x4 v{};
                    if (xchunk + 8 <= left) {
                        __builtin_memcpy(&v, xp[u] + n + xchunk, 16);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (xchunk + i < left) v[i / 2] |= (uint32_t)xp[u][n + xchunk + i] << (16 * (i & 1));
                    }
                    reinterpret_cast<u32x4*>(l)[lane] = v;
                }
            }
            const Rsrc wr = make_rsrc(wt.W + n * row_bytes + k0 / 2, left ? left * row_bytes - k0 / 2 : 0);
#pragma unroll
            for (int u = 0; u < WI; ++u) {
                const int r = 8 * (wave + 4 * u) + (lane >> 3);
                const int chunk = 16 * ((lane & 7) ^ (2 * ((r >> 3) & 3)));
                copy16(wr, within((uint32_t)(r * row_bytes) + chunk, chunk, (int)(K - k0 < BN ? K - k0 : BN) / 2),
                       d + XB + (wave + 4 * u) * 1024);
            }
        };
        // Scales: lane l has row n + l of the stage; as 512 s and -z s in LDS, [group][row].
        float* panel = reinterpret_cast<float*>(smem + STAGES * STAGE + wave * SCALES);
        const int64_t kw = k0 + 64 * wave < K ? k0 + 64 * wave : K - 1;  // (columns past K are not stored)
        const int64_t g0 = kw / wt.group, g1 = wt.group == 32 && g0 + 1 < KG ? g0 + 1 : g0;
        struct Scale {
            uint32_t s[2], z[2];
        };
        auto load_scales = [&](int s, Scale& c) {
            const int64_t n = (int64_t)s * BK + lane;
            const bool in = n < N;
            const int64_t at = (in ? n : 0) * KG;
            c.s[0] = in ? wt.scales[at + g0] : 0u;
            c.s[1] = in ? wt.scales[at + g1] : 0u;
            c.z[0] = wt.zeros ? wt.zeros[at + g0] & 15u : 8u;
            c.z[1] = wt.zeros ? wt.zeros[at + g1] & 15u : 8u;
        };
        auto put_scales = [&](int s, const Scale& c) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float f = scale_f32(c.s[g], wt.s_f16);
                float* p = panel + ((s & 1) * 2 + g) * (2 * BK) + 2 * lane;
                p[0] = 512.0f * f;
                p[1] = -(float)c.z[g] * f;
            }
        };
        f32x4 acc[4][MT];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[t][j] = f32x4{};
        const int p0 = gqf8::pos128(fr, fq), p1 = gqf8::pos128(fr, 4 + fq);
        // lane: columns 64 wave + 4 fr .. + 3 (two bytes), rows 32 h + 8 fq .. + 7
        const int wat = (8 * fq) * 128 + ((wave ^ fq) * 32) + 2 * fr;
        const int gsel = wt.group == 32 ? fr >> 3 : 0;
        Scale sc;
        if (S > 0) {
            load_scales(0, sc);
#pragma unroll
            for (int s = 0; s < STAGES; ++s) load(s);
            put_scales(0, sc);
            load_scales(1, sc);
        }
        for (int s = 0; s < S; ++s) {
            if constexpr (DMA) wait_copies<(STAGES - 1) * (XI + WI)>();
            else wait_copies<0>();
            gqd::lds_barrier();
            const uint8_t* d = smem + (s % STAGES) * STAGE;
            const u32x4* xd = reinterpret_cast<const u32x4*>(d);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                typename T::x8 b[MT];
#pragma unroll
                for (int j = 0; j < MT; ++j) b[j] = __builtin_bit_cast(typename T::x8, xd[128 * j + (h ? p1 : p0)]);
                const uint8_t* wd = d + XB + 32 * h * 128 + wat;
                const f32x4* sp = reinterpret_cast<const f32x4*>(panel + ((s & 1) * 2 + gsel) * (2 * BK) +
                                                                 2 * (32 * h + 8 * fq));
                u32x4 a[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = (uint32_t)*reinterpret_cast<const uint16_t*>(wd + 256 * i) |
                                       (uint32_t)*reinterpret_cast<const uint16_t*>(wd + 256 * i + 128) << 16;
                    const int lo = (int)(w & 0x0f0f0f0fu), hi = (int)((w >> 4) & 0x0f0f0f0fu);
                    const f32x4 f = sp[i];  // (512 s, -z s) of rows 2 i, 2 i + 1
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
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[t][j] = T::mfma(__builtin_bit_cast(typename T::x8, a[t]), b[j], acc[t][j]);
            }
            put_scales(s + 1, sc);
            load_scales(s + 2, sc);
            gqd::lds_barrier();
            load(s + STAGES);
        }
        wait_copies<0>();
        // lane: columns 64 wave + 16 fq .. + 15 of row 16 j + fr: 4 r + t
        const int64_t k = k0 + 64 * wave + 16 * fq;
        if (k >= K) return;  // (K is a multiple of 32)
        const bool vec = (lddx & 7) == 0;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row = 16 * j + fr;
            if (row >= rows) continue;
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

template <typename T, int MT, bool DMA>
__global__ __launch_bounds__(256, 2) void k_g4_dx(G4Weights wt, Rows a, int gm, int gn) {
    using U = Tile<T, MT, DMA>;
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
    U::run(of_expert(wt, t.e), a.dY + t.row0 * a.lddy, a.lddy, t.rows, a.dX + t.row0 * a.lddx, a.lddx,
           (int64_t)tn * BN, smem);
}

template <typename T, int MT, bool DMA>
hipError_t launch(const G4Weights& w, const Rows& a, hipStream_t s) {
    using U = Tile<T, MT, DMA>;
    const int64_t gm = a.offsets ? most_tiles(a.M, a.n_experts, U::BM) : (a.M + U::BM - 1) / U::BM;
    const int64_t gn = (w.K + BN - 1) / BN;
    if (!grid_ok(gm * gn, 256)) return hipErrorInvalidValue;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_g4_dx<T, MT, DMA>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, U::BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_g4_dx<T, MT, DMA>), dim3((unsigned)(gm * gn)), dim3(256), U::BYTES, s, w, a, (int)gm,
                       (int)gn);
    return hipGetLastError();
}

template <typename T, bool DMA>
hipError_t launch(const G4Weights& w, const Rows& a, hipStream_t s) {
    const int64_t per = a.M / a.n_experts;  // rows an expert has
    if (per <= 32) return launch<T, 2, DMA>(w, a, s);
    if (per <= 64) return launch<T, 4, DMA>(w, a, s);
    return launch<T, 8, DMA>(w, a, s);
}

template <typename T>
hipError_t launch(const G4Weights& w, const Rows& a, hipStream_t s) {
    return w.N % 8 == 0 && a.lddy % 8 == 0 ? launch<T, true>(w, a, s) : launch<T, false>(w, a, s);
}

}  // namespace

hipError_t gqk_g4_matmul_dx(const G4Weights& w, const void* dY, int dtype, int64_t M, int64_t lddy, void* dX,
                            int64_t lddx, int n_experts, const int32_t* offsets, hipStream_t s) {
    const Rows a{static_cast<const uint16_t*>(dY), M, lddy, static_cast<uint16_t*>(dX), lddx, n_experts, offsets};
    return dtype == gqd::DT_BF16 ? launch<Bf16>(w, a, s) : launch<F16>(w, a, s);
}
