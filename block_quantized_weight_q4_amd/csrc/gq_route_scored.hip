// gq_route_scored.hip -- per-token expert routing by scores (softmax or
// sigmoid) with a selection bias and groups, in one launch (gfx950, wave64).
//
// Mathematics: c[e] = s[e] + bias[e]; a group's value is its largest c or the
// sum of its two largest; the experts of the best top_groups groups compete
// for the top_k places by c; the weights are the chosen s, renormalised and
// scaled.  Everything that decides is held in 64 bits: two fp32 sigmoids of
// neighbouring experts round to the same or the wrong order about once in
// 10^4 tokens, and a choice once made is not a rounding error any more.  The
// vector unit's fp64 rate equals its fp32 rate here, so this costs only the
// longer exp.
//
// One wavefront per token.  Lane l holds the experts l NI .. l NI + NI - 1
// (blocked, so that the lowest lane that holds the largest value also holds
// the lowest expert id among equals) as order-preserving 64-bit images of c;
// a wave maximum of the images' upper halves by DPP, a ballot and a readlane find
// each place, the lower halves only where the upper ones are equal.  The scores
// wait in LDS for the places that take them.
// Bound by latency: T x E logits are a few megabytes at most.  Measured: one
// token of 256 experts in 8 groups 5.2 us, 3015 tokens of 128 experts 6.1 us (6.2
// and 8.1 with 64-bit maxima and the chosen scores computed again).  Above 1024
// experts a lane holds 64, whose scores fill the registers of a SIMD: one wavefront
// each, one token of 2048 experts 35 us, 3015 of them 122 us (1024: 10.5 and 25 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gq_device.h"
#include "gq_f8_internal.h"

namespace {

constexpr int GROUP_TOP2 = 1, SCORE_SIGMOID = 1;

// Orders fences of one wavefront's own LDS traffic: its lanes exchange values
// through LDS that no other wavefront touches.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
    __builtin_amdgcn_wave_barrier();
}

// fp64 -> 64-bit key with the same order; NaN is taken as -inf.  No real key is 0.
__device__ __forceinline__ uint64_t order_key64(double v) {
    if (v != v) v = -__builtin_inf();
    v += 0.0;  // -0 -> +0
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// Largest value of the wave, in every lane: each step is one instruction (0,
// which lanes without a source get, is the smallest value).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max_of<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8: each row's maximum in its last lane
    v = max_of<0x112, 0xF>(v);
    v = max_of<0x114, 0xF>(v);
    v = max_of<0x118, 0xF>(v);
    v = max_of<0x142, 0xA>(v);  // row_bcast15 into rows 1 and 3
    v = max_of<0x143, 0xC>(v);  // row_bcast31 into rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The lowest lane that holds the largest key: by the upper halves, and by the
// lower ones where those are equal.
__device__ __forceinline__ int wave_argmax_u64(uint64_t v) {
    const uint32_t hi = (uint32_t)(v >> 32), top = wave_max_u32(hi);
    uint64_t at = __ballot(hi == top);
    if (at & (at - 1)) {
        const uint32_t lo = hi == top ? (uint32_t)v : 0u;
        const uint32_t low = wave_max_u32(lo);
        at &= __ballot(lo == low);
    }
    return __builtin_ctzll(at);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
    if constexpr (sizeof(T) == 4) return *p;
    else return gqd::bf2f(*p);
}

// Softmax numerator or sigmoid of one logit, in fp64.
__device__ __forceinline__ double score_of(int score, float l, double m) {
    if (score == SCORE_SIGMOID) return 1.0 / (1.0 + exp(-(double)l));
    return l == -__builtin_inff() ? 0.0 : exp((double)l - m);
}

template <int NI, int WAVES, typename T>
__global__ __launch_bounds__(64 * WAVES) void k_route_scored(const T* __restrict__ logits, int n_tokens,
                                                             int n_experts, int top_k, int score,
                                                             const float* __restrict__ bias, int n_groups,
                                                             int top_groups, int group_rank, int renorm, float scale,
                                                             int32_t* __restrict__ ids, float* __restrict__ weights) {
    __shared__ double lds[WAVES][NI * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * WAVES + wave;
    if (t >= n_tokens) return;  // t is the same for the whole wave, and no barrier follows
    const T* l = logits + (int64_t)t * n_experts;
    const int e0 = lane * NI;

    // every load is unconditional, from a clamped index
    float v[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = load_logit(l + (e0 + i < n_experts ? e0 + i : n_experts - 1));
    float b[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) b[i] = bias ? bias[e0 + i < n_experts ? e0 + i : n_experts - 1] : 0.0f;
    double m = 0.0;
    if (score != SCORE_SIGMOID) {
        float mx = v[0];  // (a clamped index repeats a real logit)
#pragma unroll
        for (int i = 1; i < NI; ++i) mx = fmaxf(mx, v[i]);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
        m = mx;
    }
    double s[NI];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        s[i] = score_of(score, v[i], m);
        sum += e0 + i < n_experts ? s[i] : 0.0;
    }
    if (score != SCORE_SIGMOID) {
        const double total = wave_sum_f64(sum);
#pragma unroll
        for (int i = 0; i < NI; ++i) s[i] = s[i] == 0.0 ? 0.0 : s[i] / total;
    }
    uint64_t key[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) key[i] = e0 + i < n_experts ? order_key64(s[i] + (double)b[i]) : 0ull;

    if (n_groups > 1) {
        const int gs = n_experts / n_groups;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const double c = s[i] + (double)b[i];
            lds[wave][e0 + i] = c != c ? -__builtin_inf() : c;
        }
        wave_lds_fence();
        // P lanes per group find its two largest values
        const int P = 1 << (31 - __builtin_clz(64 / n_groups));
        const int g = lane / P;
        double a1 = -__builtin_inf(), a2 = -__builtin_inf();
        if (g < n_groups)
            for (int j = lane & (P - 1); j < gs; j += P) {
                const double x = lds[wave][g * gs + j];
                a2 = fmax(a2, fmin(a1, x));
                a1 = fmax(a1, x);
            }
        for (int off = P >> 1; off >= 1; off >>= 1) {
            const double b1 = __shfl_xor(a1, off, 64), b2 = __shfl_xor(a2, off, 64);
            a2 = fmax(fmin(a1, b1), fmax(a2, b2));
            a1 = fmax(a1, b1);
        }
        const double value = group_rank == GROUP_TOP2 && gs > 1 ? a1 + a2 : a1;
        const uint64_t gk = order_key64(value);
        // a group's rank: how many groups are ahead of it
        int rank = 0;
        for (int h = 0; h < n_groups; ++h) {
            const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(gk >> 32), h * P) << 32) |
                               (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)gk, h * P);
            rank += o > gk || (o == gk && h < g);
        }
        const uint64_t kept = __ballot(g < n_groups && rank < top_groups);  // bit h P: group h stays
        int ge = e0 / gs, r = e0 - ge * gs;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if (!((kept >> ((ge * P) & 63)) & 1ull)) key[i] = 0ull;
            if (++r == gs) {
                r = 0;
                ++ge;
            }
        }
    }

    // the scores, for whichever lane's place takes them
    wave_lds_fence();
#pragma unroll
    for (int i = 0; i < NI; ++i) lds[wave][e0 + i] = s[i];
    wave_lds_fence();

    int my_id = 0;
    for (int j = 0; j < top_k; ++j) {
        uint64_t best = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < NI; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        const int owner = wave_argmax_u64(best);
        const int e = owner * NI + __builtin_amdgcn_readlane(bi, owner);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (e == e0 + i) key[i] = 0ull;
        if (lane == j) my_id = e;
    }
    if (my_id >= n_experts) my_id = n_experts - 1;  // (cannot happen: enough experts stay)
    const double chosen_s = lane < top_k ? lds[wave][my_id] : 0.0;
    double w = chosen_s;
    if (renorm) {
        const double chosen = wave_sum_f64(chosen_s);
        w = chosen == 0.0 ? 0.0 : chosen_s / chosen;
    }
    if (lane < top_k) {
        ids[(int64_t)t * top_k + lane] = my_id;
        weights[(int64_t)t * top_k + lane] = (float)(w * (double)scale);
    }
}

struct Args {
    const void* logits;
    int dtype, n_tokens, n_experts, top_k, score;
    const float* bias;
    int n_groups, top_groups, group_rank, renorm;
    float scale;
    int32_t* ids;
    float* weights;
};

template <int NI, typename T>
hipError_t launch_t(const Args& a, hipStream_t s) {
    constexpr int WAVES = NI <= 16 ? 4 : 1;  // at most 32 KB of LDS
    const unsigned grid = (unsigned)((a.n_tokens + (int64_t)WAVES - 1) / WAVES);
    hipLaunchKernelGGL((k_route_scored<NI, WAVES, T>), dim3(grid), dim3(64 * WAVES), 0, s,
                       static_cast<const T*>(a.logits), a.n_tokens, a.n_experts, a.top_k, a.score, a.bias, a.n_groups,
                       a.top_groups, a.group_rank, a.renorm, a.scale, a.ids, a.weights);
    return hipGetLastError();
}

template <int NI>
hipError_t launch(const Args& a, hipStream_t s) {
    return a.dtype == gqd::DT_F32 ? launch_t<NI, float>(a, s) : launch_t<NI, uint16_t>(a, s);
}

}  // namespace

hipError_t gqk_route_scored(const void* logits, int dtype, int n_tokens, int n_experts, int top_k, int score,
                            const float* bias, int n_groups, int top_groups, int group_rank, int renorm, float scale,
                            int32_t* ids, float* weights, hipStream_t s) {
    const Args a{logits, dtype, n_tokens, n_experts, top_k, score, bias, n_groups, top_groups, group_rank, renorm,
                 scale, ids, weights};
    const int ni = (n_experts + 63) / 64;
    if (ni <= 1) return launch<1>(a, s);
    if (ni <= 2) return launch<2>(a, s);
    if (ni <= 4) return launch<4>(a, s);
    if (ni <= 8) return launch<8>(a, s);
    if (ni <= 16) return launch<16>(a, s);
    return launch<64>(a, s);
}
