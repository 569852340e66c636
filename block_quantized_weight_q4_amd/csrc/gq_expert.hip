// gq_expert.hip -- tokens sorted by expert and back, and their gradients
// (gfx950).  All are bound by HBM where there are many rows, and by the launch
// where there are few.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "gq_device.h"
#include "gq_expert_internal.h"

using gqd::u32x4;

namespace {

constexpr int MAX_E = 4096;

// ------------------------------------------------------------------ sort ----

// Workgroup b places the slots [b * chunk, (b + 1) * chunk) (chunk a multiple of
// 64).  Each counts all the slots by itself, those before its own apart from the
// others, so that no workgroup waits for another and one launch does it: the ids
// are few bytes and come from the caches.  Then it scans the experts, and its
// wavefronts place their slots one after another: equal ids of a wavefront find
// each other by a ballot for each bit of the id.  3015 x 8 slots: 7.5 us; 1,048,576 slots
// 80 to 106 us, bound by every workgroup's reading all 4 MB of ids from its L2 and counting
// them in LDS (counts of a launch before would halve that, and make every routing two).
template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_sort(const int32_t* __restrict__ ids, int S, int E, int chunk,
                                                  int32_t* __restrict__ offsets, int32_t* __restrict__ place) {
    constexpr int WAVES = THREADS / 64;
    __shared__ int before[MAX_E], rest[MAX_E];  // slots before this workgroup's, the others; then places
    __shared__ int wave_sum[WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int first = blockIdx.x * chunk;
    for (int e = tid; e < E; e += THREADS) before[e] = rest[e] = 0;
    __syncthreads();
    constexpr int U = 8;  // loads on their way at once
    for (int s0 = 0; s0 < S; s0 += U * 4 * THREADS) {
        int4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + (u * THREADS + tid) * 4;
            v[u] = make_int4(-1, -1, -1, -1);
            if (s + 4 <= S) {
                v[u] = *reinterpret_cast<const int4*>(ids + s);  // (ids are 16-byte aligned)
            } else {
                if (s < S) v[u].x = ids[s];
                if (s + 1 < S) v[u].y = ids[s + 1];
                if (s + 2 < S) v[u].z = ids[s + 2];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + (u * THREADS + tid) * 4;
            if (s0 + u * THREADS * 4 >= S) break;
            int* count = s < first ? before : rest;  // (first is a multiple of 4)
            if ((unsigned)v[u].x < (unsigned)E) atomicAdd(&count[v[u].x], 1);
            if ((unsigned)v[u].y < (unsigned)E) atomicAdd(&count[v[u].y], 1);
            if ((unsigned)v[u].z < (unsigned)E) atomicAdd(&count[v[u].z], 1);
            if ((unsigned)v[u].w < (unsigned)E) atomicAdd(&count[v[u].w], 1);
        }
    }
    __syncthreads();
    // exclusive sums over the experts, a thread a run of them
    const int per = (E + THREADS - 1) / THREADS;
    const int lo = tid * per < E ? tid * per : E, hi = lo + per < E ? lo + per : E;
    int n = 0;
    for (int e = lo; e < hi; ++e) n += before[e] + rest[e];
    int incl = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(incl, off, 64);
        if (lane >= off) incl += v;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int sum = incl - n;
    for (int w = 0; w < wave; ++w) sum += wave_sum[w];
    for (int e = lo; e < hi; ++e) {
        const int here = before[e] + rest[e];
        if (blockIdx.x == 0) offsets[e] = sum;
        before[e] += sum;  // the place of this workgroup's first slot of e
        sum += here;
    }
    if (blockIdx.x == 0 && tid == THREADS - 1) offsets[E] = sum;
    __syncthreads();
    const int last = first + chunk < S ? first + chunk : S;
    for (int s0 = first; s0 < last; s0 += THREADS) {
        const int s = s0 + tid, id = s < last ? ids[s] : -1;
        const bool ok = (unsigned)id < (unsigned)E;
        uint64_t same = __ballot(ok);
#pragma unroll
        for (int b = 0; b < 12; ++b) {  // (E <= 4096)
            const uint64_t m = __ballot((id >> b) & 1);
            same &= (id >> b) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1)), count = __popcll(same);
        const int waves = (last - s0 + 63) / 64 < WAVES ? (last - s0 + 63) / 64 : WAVES;
        for (int w = 0; w < waves; ++w) {
            if (wave == w) {
                const int base = ok ? before[id] : 0;
                if (ok && rank == count - 1) before[id] = base + count;  // (behind the reads of the others)
                if (s < last) place[s] = ok ? base + rank : -1;
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------ rows ----

// Element types of rows; V of them are 16 bytes.
struct F32 {
    static constexpr int V = 4;
    typedef uint32_t elem;
    static __device__ __forceinline__ float get(const u32x4& v, int i) {
        const uint32_t u = v[i];  // (a copy first: a bit_cast of a vector's element takes element 0)
        return __builtin_bit_cast(float, u);
    }
    static __device__ __forceinline__ uint32_t narrow(float f) { return __builtin_bit_cast(uint32_t, f); }
};
struct Half16 {
    static constexpr int V = 8;
    typedef uint16_t elem;
    static __device__ __forceinline__ uint16_t bits(const u32x4& v, int i) {
        return (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
};
struct Bf16 : Half16 {
    static __device__ __forceinline__ float get(const u32x4& v, int i) {
        const uint32_t u = i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16;
        return __builtin_bit_cast(float, u);
    }
    static __device__ __forceinline__ uint16_t narrow(float f) { return gqd::f2bf(f); }
};
struct F16 : Half16 {
    static __device__ __forceinline__ float get(const u32x4& v, int i) { return gqd::h2f(bits(v, i)); }
    static __device__ __forceinline__ uint16_t narrow(float f) { return gqd::f2h(f); }
};

// 16 bytes of a row from p, of whose elements `left` are the row's (the others zeros,
// not read, not written); rows start at any element, which vector memory instructions
// allow.  (The asm keeps the two ways apart, which would else share narrow loads.)
template <typename E>
__device__ __forceinline__ u32x4 read16(const E* p, int64_t left) {
    constexpr int N = 16 / sizeof(E);
    u32x4 v{};
    if (left >= N) {
        __builtin_memcpy(&v, p, 16);
    } else {
        __asm__ volatile("" : "+v"(p));
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) v[i * sizeof(E) / 4] |= (uint32_t)p[i] << (i * sizeof(E) % 4 * 8);
    }
    return v;
}
template <typename E>
__device__ __forceinline__ void write16(E* p, int64_t left, const u32x4& v) {
    constexpr int N = 16 / sizeof(E);
    if (left >= N) {
        __builtin_memcpy(p, &v, 16);
    } else {
        __asm__ volatile("" : "+v"(p));
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = (E)(v[i * sizeof(E) / 4] >> (i * sizeof(E) % 4 * 8));
    }
}
// N values as type T from p on.
template <typename T, int N>
__device__ __forceinline__ void write_as(typename T::elem* p, int64_t left, const float (&f)[N]) {
#pragma unroll
    for (int k = 0; k < N; k += T::V) {
        u32x4 v{};
#pragma unroll
        for (int i = 0; i < T::V; ++i)
            v[i * 4 / T::V] |= (uint32_t)T::narrow(f[k + i]) << (T::V == 8 ? 16 * (i & 1) : 0);
        if (k < left) write16(p + k, left - k, v);
    }
}

// The row of slot s, -1 if it has none.
__device__ __forceinline__ int64_t row_of(const int32_t* __restrict__ place, int64_t s, int64_t S) {
    const int64_t p = place[s];
    return p >= 0 && p < S ? p : -1;
}

// A wavefront's pieces of 1 KB of the tokens' rows, `pieces` a row: f(t, d) with the
// token and this lane's first element.
template <int V, typename F>
__device__ __forceinline__ void each_piece(int n_tokens, int64_t D, int64_t pieces, F f) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < pieces * n_tokens; i += (int64_t)gridDim.x * 4) {
        const int64_t t = i / pieces, d = ((i - t * pieces) * 64 + (threadIdx.x & 63)) * V;
        if (d < D) f(t, d);
    }
}

// Copies each piece to the places of the token's slots.  3015 x 8 slots of 2816 bf16 (153
// MB): 31 us, the rate of a large copy.
template <typename T>
__global__ __launch_bounds__(256) void k_gather(const typename T::elem* __restrict__ x, int n_tokens, int top_k,
                                                int64_t D, int64_t ldx, const int32_t* __restrict__ place,
                                                typename T::elem* __restrict__ xs, int64_t ldxs, int64_t pieces) {
    const int64_t S = (int64_t)n_tokens * top_k;
    each_piece<T::V>(n_tokens, D, pieces, [&](int64_t t, int64_t d) {
        const u32x4 v = read16(x + t * ldx + d, D - d);
#pragma unroll 8
        for (int j = 0; j < top_k; ++j) {
            const int64_t p = row_of(place, t * top_k + j, S);
            if (p >= 0) write16(xs + p * ldxs + d, D - d, v);
        }
    });
}

// Adds up a piece of the token's slots' rows, in their order.  3015 x 8 slots of 2816 bf16
// (153 MB): 31 us, 4.9 TB/s.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void k_combine(const typename T::elem* __restrict__ ys, int n_tokens, int top_k,
                                                 int64_t D, int64_t ldys, const int32_t* __restrict__ place,
                                                 const float* __restrict__ w, typename Y::elem* __restrict__ y,
                                                 int64_t ldy, int64_t pieces) {
    const int64_t S = (int64_t)n_tokens * top_k;
    each_piece<T::V>(n_tokens, D, pieces, [&](int64_t t, int64_t d) {
        float sum[T::V];
#pragma unroll
        for (int e = 0; e < T::V; ++e) sum[e] = 0.0f;
        constexpr int U = 8;  // rows on their way at once
        for (int j0 = 0; j0 < top_k; j0 += U) {
            u32x4 v[U];
            float f[U];
            bool ok[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u < top_k ? j0 + u : top_k - 1;
                const int64_t p = row_of(place, t * top_k + j, S);
                ok[u] = p >= 0 && j0 + u < top_k;
                f[u] = w ? w[t * top_k + j] : 1.0f;
                if (ok[u]) v[u] = read16(ys + p * ldys + d, D - d);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (ok[u]) {
#pragma unroll
                    for (int e = 0; e < T::V; ++e) sum[e] = __builtin_fmaf(f[u], T::get(v[u], e), sum[e]);
                }
        }
        write_as<Y>(y + t * ldy + d, D - d, sum);
    });
}

// A workgroup has one token, its four wavefronts 1 KB pieces of the row in turn.
// (dys may be ys: no __restrict__, and a piece is read before it is written)
// 3015 x 8 slots of 2816 bf16 (289 MB): 64 us, 4.5 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void k_combine_grad(const typename T::elem* __restrict__ dy, int n_tokens,
                                                      int top_k, int64_t D, int64_t lddy, const typename T::elem* ys,
                                                      int64_t ldys, const int32_t* __restrict__ place,
                                                      const float* __restrict__ w, typename T::elem* dys,
                                                      int64_t lddys, float* __restrict__ dw) {
    constexpr int U = 8;  // slots at a time
    __shared__ float part[4][U];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = blockIdx.x, S = (int64_t)n_tokens * top_k;
    for (int j0 = 0; j0 < top_k; j0 += U) {
        int64_t p[U];
        float f[U], sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u < top_k ? j0 + u : top_k - 1;
            p[u] = j0 + u < top_k ? row_of(place, t * top_k + j, S) : -1;
            f[u] = w ? w[t * top_k + j] : 1.0f;
            sum[u] = 0.0f;
        }
        for (int64_t d = ((int64_t)wave * 64 + lane) * T::V; d < D; d += 256 * T::V) {
            const u32x4 g = read16(dy + t * lddy + d, D - d);
            u32x4 v[U];
            if (dw) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (p[u] >= 0) v[u] = read16(ys + p[u] * ldys + d, D - d);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p[u] < 0) continue;
                if (dw) {
#pragma unroll
                    for (int e = 0; e < T::V; ++e) sum[u] = __builtin_fmaf(T::get(g, e), T::get(v[u], e), sum[u]);
                }
                if (dys) {
                    typename T::elem* q = dys + p[u] * lddys + d;
                    if (w) {
                        float out[T::V];
#pragma unroll
                        for (int e = 0; e < T::V; ++e) out[e] = f[u] * T::get(g, e);
                        write_as<T>(q, D - d, out);
                    } else {
                        write16(q, D - d, g);
                    }
                }
            }
        }
        if (!dw) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) sum[u] += __shfl_xor(sum[u], off, 64);
            if (lane == 0) part[wave][u] = sum[u];
        }
        __syncthreads();
        const int u = threadIdx.x;
        if (u < U && j0 + u < top_k)
            dw[t * top_k + j0 + u] = (part[0][u] + part[1][u]) + (part[2][u] + part[3][u]);
        __syncthreads();
    }
}

template <typename T>
int64_t pieces_of(int64_t D) {
    return (D + 64 * T::V - 1) / (64 * T::V);
}

// (a launch has at most 2^32 threads: beyond, the workgroups go round again)
dim3 grid_of(int64_t pieces) {
    constexpr int64_t MOST = (int64_t)1 << 23;
    return dim3((unsigned)((pieces + 3) / 4 < MOST ? (pieces + 3) / 4 : MOST));
}

template <typename T>
hipError_t gather(const void* x, int n_tokens, int top_k, int64_t D, int64_t ldx, const int32_t* place, void* xs,
                  int64_t ldxs, hipStream_t s) {
    using E = typename T::elem;
    const int64_t pieces = pieces_of<T>(D);
    hipLaunchKernelGGL(k_gather<T>, grid_of(pieces * n_tokens), dim3(256), 0, s, static_cast<const E*>(x), n_tokens,
                       top_k, D, ldx, place, static_cast<E*>(xs), ldxs, pieces);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t combine(const void* ys, int n_tokens, int top_k, int64_t D, int64_t ldys, const int32_t* place,
                   const float* w, void* y, int64_t ldy, hipStream_t s) {
    const int64_t pieces = pieces_of<T>(D);
    hipLaunchKernelGGL((k_combine<T, Y>), grid_of(pieces * n_tokens), dim3(256), 0, s,
                       static_cast<const typename T::elem*>(ys), n_tokens, top_k, D, ldys, place, w,
                       static_cast<typename Y::elem*>(y), ldy, pieces);
    return hipGetLastError();
}

template <typename T>
hipError_t combine_grad(const void* dy, int n_tokens, int top_k, int64_t D, int64_t lddy, const void* ys,
                        int64_t ldys, const int32_t* place, const float* w, void* dys, int64_t lddys, float* dw,
                        hipStream_t s) {
    using E = typename T::elem;
    hipLaunchKernelGGL(k_combine_grad<T>, dim3(n_tokens), dim3(256), 0, s, static_cast<const E*>(dy), n_tokens, top_k,
                       D, lddy, static_cast<const E*>(ys), ldys, place, w, static_cast<E*>(dys), lddys, dw);
    return hipGetLastError();
}

}  // namespace

hipError_t gqk_expert_sort(const int32_t* ids, int n_tokens, int top_k, int n_experts, int32_t* offsets,
                           int32_t* place, hipStream_t s) {
    const int S = n_tokens * top_k;
    if (S <= 1024) {
        hipLaunchKernelGGL(k_sort<256>, dim3(1), dim3(256), 0, s, ids, S, n_experts, 1024, offsets, place);
        return hipGetLastError();
    }
    int chunk = (S / 256 + 63) / 64 * 64;  // about a workgroup a CU
    if (chunk < 256) chunk = 256;
    hipLaunchKernelGGL(k_sort<1024>, dim3((S + chunk - 1) / chunk), dim3(1024), 0, s, ids, S, n_experts, chunk, offsets,
                       place);
    return hipGetLastError();
}

hipError_t gqk_expert_gather(const void* x, int dtype, int n_tokens, int top_k, int64_t D, int64_t ldx,
                             const int32_t* place, void* xs, int64_t ldxs, hipStream_t s) {
    if (dtype == gqd::DT_F32) return gather<F32>(x, n_tokens, top_k, D, ldx, place, xs, ldxs, s);
    return gather<Bf16>(x, n_tokens, top_k, D, ldx, place, xs, ldxs, s);  // (a copy: any 16 bits)
}

hipError_t gqk_expert_combine(const void* ys, int dtype, int n_tokens, int top_k, int64_t D, int64_t ldys,
                              const int32_t* place, const float* w, void* y, int y_dtype, int64_t ldy,
                              hipStream_t s) {
    if (dtype == gqd::DT_F32) return combine<F32, F32>(ys, n_tokens, top_k, D, ldys, place, w, y, ldy, s);
    if (dtype == gqd::DT_BF16)
        return y_dtype == gqd::DT_F32 ? combine<Bf16, F32>(ys, n_tokens, top_k, D, ldys, place, w, y, ldy, s)
                                      : combine<Bf16, Bf16>(ys, n_tokens, top_k, D, ldys, place, w, y, ldy, s);
    return y_dtype == gqd::DT_F32 ? combine<F16, F32>(ys, n_tokens, top_k, D, ldys, place, w, y, ldy, s)
                                  : combine<F16, F16>(ys, n_tokens, top_k, D, ldys, place, w, y, ldy, s);
}

hipError_t gqk_expert_combine_grad(const void* dy, int dtype, int n_tokens, int top_k, int64_t D, int64_t lddy,
                                   const void* ys, int64_t ldys, const int32_t* place, const float* w, void* dys,
                                   int64_t lddys, float* dw, hipStream_t s) {
    if (dtype == gqd::DT_F32)
        return combine_grad<F32>(dy, n_tokens, top_k, D, lddy, ys, ldys, place, w, dys, lddys, dw, s);
    if (dtype == gqd::DT_BF16)
        return combine_grad<Bf16>(dy, n_tokens, top_k, D, lddy, ys, ldys, place, w, dys, lddys, dw, s);
    return combine_grad<F16>(dy, n_tokens, top_k, D, lddy, ys, ldys, place, w, dys, lddys, dw, s);
}
