// select.cu -- the choice of experts from router logits: softmax, sigmoid or
// sqrt-softplus scores, a bias for the choice, groups of experts, top-k,
// weights with or without renormalisation.
//
//   s_e = score(z_e),  c_e = s_e (+ score_bias[e])
//   group score = max c, or the sum of the two largest c, of its experts
//   the topk_group best groups stay; the k largest c in them are chosen
//   w_j = scale * s_j (/ sum of the chosen s)
//
// One warp per token: lane l holds the experts l, l + 32, ... (E <= 256). The
// choice is k rounds of a warp-wide argmax on order-preserving integer keys.
//
// Ranking. The scores increase with the logit, so without a bias the experts
// are ranked by the logits themselves, exactly. With a bias, and for sums of
// two scores, the values are computed in fp32 and every comparison that decides
// something (consecutive choices, the first expert left out, the last group
// kept against the best one dropped) has to be wider than the evaluation's
// error bound; a token where one is not runs once more in fp64 (about one token
// in 500 at E = 256). fp64 for every token would take the fp64 pipe several
// times longer than reading the logits takes.
//
// Bound: the logits, 4 T E bytes, against about 500 instructions per token.
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int WARPS = 4;      // tokens per CTA
constexpr int Q = 8;          // experts per lane
constexpr int PAD_E = 256 + 8;

struct SelectArgs {
    const float* logits;
    long ld;
    const float* bias;
    int score_fn, n_group, topk_group, group_score, renorm;
    int T, E, k;
    float scale;
    int* idx;
    float* w;
};

// NaN -> -inf (out of the choice), +inf -> the largest finite float.
__device__ __forceinline__ float cleaned(float v) { return v != v ? -INFINITY : fminf(v, FLT_MAX); }

// Order-preserving keys: a larger value has a larger key; 0 is no value's key.
__device__ __forceinline__ uint32_t key_of(float v) { return order_key(v); }
__device__ __forceinline__ float value_of(uint32_t k) { return key_value(k); }
__device__ __forceinline__ unsigned long long key_of(double v) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ double value_of(unsigned long long k) {
    return __longlong_as_double((long long)((k >> 63) ? (k ^ (1ull << 63)) : ~k));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t k) {
    return __reduce_max_sync(0xffffffffu, k);
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long p = __shfl_xor_sync(0xffffffffu, k, o);
        k = p > k ? p : k;
    }
    return k;
}
template <typename V>
__device__ __forceinline__ V warp_max_value(V v) { return value_of(warp_max(key_of(v))); }

__device__ __forceinline__ float warp_total(float v) { return warp_sum(v); }
__device__ __forceinline__ double warp_total(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Scores (softmax: before the division by the sum; z - max for z). Errors of
// the fp32 forms are below 1e-6 of 1 + score: the fast exponential is within
// |z| 2^-24 + 2^-22 of its value, which the score's slope in z turns into at
// most that.
__device__ __forceinline__ float score_of(float z, int fn) {
    if (fn == MOE_SCORE_SOFTMAX) return __expf(z);
    if (fn == MOE_SCORE_SQRT_SOFTPLUS)
        return sqrtf(fmaxf(z, 0.f) + log1pf(__expf(-fabsf(z))));
    return __fdividef(1.0f, 1.0f + __expf(-z));
}
__device__ __noinline__ double score_of(double z, int fn) {
    if (fn == MOE_SCORE_SOFTMAX) return exp(z);
    if (fn == MOE_SCORE_SQRT_SOFTPLUS) return sqrt(fmax(z, 0.0) + log1p(exp(-fabs(z))));
    return 1.0 / (1.0 + exp(-z));
}

// Whether a > b can be told apart in spite of the evaluation's error (fp64:
// always taken as it is; two -infinities are a tie that the index decides).
__device__ __forceinline__ bool decided(float a, float b) {
    return b == -INFINITY || a - b > 4e-6f * (1.0f + fmaxf(fabsf(a), fabsf(b)));
}
__device__ __forceinline__ bool decided(double, double) { return true; }

template <typename V>
struct Scratch {
    V value[PAD_E];   // value of expert e at e + e / 32 (no bank conflicts between groups)
    V group[256];
    uint32_t kept[8]; // bit g: group g stays
};
union WarpScratch {
    Scratch<float> f;
    Scratch<double> d;
};

// One token's choice by one warp; lane j < k gets the j-th expert in `mine`.
// Returns whether every comparison was wider than the error (uniform).
template <typename V>
__device__ __forceinline__ bool choose(const SelectArgs& a, const float (&z)[Q], float zmax,
                                       Scratch<V>& sc, int& mine) {
    using K = decltype(key_of(V()));
    const int lane = threadIdx.x & 31;
    const bool top2 = a.n_group > 1 && a.group_score == MOE_GROUP_TOP2;
    V r[Q], c[Q];  // what experts are ranked by; what groups sum
    if (a.bias || top2) {
        V total = 1;
        if (a.score_fn == MOE_SCORE_SOFTMAX) {
            V part = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (lane + 32 * q < a.E) {
                    c[q] = score_of((V)z[q] - (V)zmax, a.score_fn);
                    part += c[q];
                }
            total = warp_total(part);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = lane + 32 * q;
            if (e >= a.E) continue;
            V s = a.score_fn == MOE_SCORE_SOFTMAX ? c[q] / total : score_of((V)z[q], a.score_fn);
            if (a.bias) s += (V)cleaned(a.bias[e]);
            c[q] = z[q] == -INFINITY ? (V)-INFINITY : s;
            r[q] = a.bias ? c[q] : (V)z[q];
        }
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) c[q] = r[q] = (V)z[q];
    }
    K key[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) key[q] = lane + 32 * q < a.E ? key_of(r[q]) : (K)0;
    bool sure = true;

    if (a.n_group > 1) {
        const int G = a.n_group, n = a.E / G;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int e = lane + 32 * q;
            if (e < a.E) sc.value[e + (e >> 5)] = c[q];
        }
        __syncwarp();
        // LP lanes per group (a power of two), groups in passes of 32 / LP
        int LP = 1;
        while (LP * 2 * G <= 32) LP *= 2;
        const int sub = lane & (LP - 1);
        for (int g0 = 0; g0 < G; g0 += 32 / LP) {
            const int g = g0 + lane / LP;
            V v1 = -INFINITY, v2 = -INFINITY;
            if (g < G)
                for (int i = sub; i < n; i += LP) {
                    const int e = g * n + i;
                    const V v = sc.value[e + (e >> 5)];
                    if (v > v1) { v2 = v1; v1 = v; } else if (v > v2) v2 = v;
                }
            for (int o = 1; o < LP; o <<= 1) {
                const V u1 = __shfl_xor_sync(0xffffffffu, v1, o);
                const V u2 = __shfl_xor_sync(0xffffffffu, v2, o);
                if (u1 > v1) { v2 = v1 > u2 ? v1 : u2; v1 = u1; } else if (u1 > v2) v2 = u1;
            }
            if (g < G && sub == 0) sc.group[g] = top2 ? v1 + v2 : v1;
        }
        __syncwarp();
        // a group stays if fewer than topk_group groups are ahead of it
        K worst_kept = ~(K)0, best_left = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            int ahead = 0;
            const V own = sc.group[g < G ? g : 0];
            for (int o = 0; o < G; ++o) {
                const V v = sc.group[o];
                ahead += v > own || (v == own && o < g);
            }
            const bool keep = g < G && ahead < a.topk_group;
            const uint32_t bits = __ballot_sync(0xffffffffu, keep);
            if (lane == 0) sc.kept[g0 >> 5] = bits;
            const K kk = key_of(own);
            if (keep) worst_kept = kk < worst_kept ? kk : worst_kept;
            if (g < G && !keep) best_left = kk > best_left ? kk : best_left;
        }
        if ((a.bias || top2) && a.topk_group < G)
            sure = decided(value_of((K)~warp_max((K)~worst_kept)), value_of(warp_max(best_left)));
        __syncwarp();
        // e / n by a multiplication: exact for e < 256 (the error e / 2^16 is
        // below the distance 1 / n >= 1 / 256 to the next integer)
        const uint32_t inv = 65536u / (uint32_t)n + 1u;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint32_t g = ((uint32_t)(lane + 32 * q) * inv) >> 16;
            if (lane + 32 * q < a.E && !((sc.kept[g >> 5] >> (g & 31u)) & 1u)) key[q] = 0;
        }
    }

    // k rounds, and where values are inexact one more for the first one left out
    const int rounds = a.bias ? a.k + 1 : a.k;
    V before = 0;
    for (int j = 0; j < rounds; ++j) {
        K best = key[0];
        int bq = 0;
#pragma unroll
        for (int q = 1; q < Q; ++q)
            if (key[q] > best) { best = key[q]; bq = q; }
        const K m = warp_max(best);
        if (m == 0) break;  // nothing left (uniform)
        const uint32_t e = __reduce_min_sync(0xffffffffu,
                                             best == m ? (uint32_t)(lane + 32 * bq) : 0xffffffffu);
        if (a.bias) {
            const V v = value_of(m);
            if (j > 0) sure = sure && decided(before, v);
            before = v;
        }
        if (lane == j) mine = (int)e;
        if ((int)(e & 31u) == lane) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if ((int)(e >> 5) == q) key[q] = 0;
        }
    }
    return sure;
}

__global__ void __launch_bounds__(WARPS * 32)
select_kernel(const SelectArgs a) {
    pdl_launch_and_wait();
    __shared__ WarpScratch scratch[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long t = (long)blockIdx.x * WARPS + warp;
    if (t >= a.T) return;
    const float* row = a.logits + t * a.ld;
    float z[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        z[q] = lane + 32 * q < a.E ? cleaned(row[lane + 32 * q]) : -INFINITY;
    float zmax = 0.f;
    if (a.score_fn == MOE_SCORE_SOFTMAX) {
        zmax = z[0];
#pragma unroll
        for (int q = 1; q < Q; ++q) zmax = fmaxf(zmax, z[q]);
        zmax = warp_max_value(zmax);
        if (zmax == -INFINITY) zmax = 0.f;  // every expert is out: all scores 0
    }
    int e = 0;
    if (!choose<float>(a, z, zmax, scratch[warp].f, e)) {
        __syncwarp();
        choose<double>(a, z, zmax, scratch[warp].d, e);
    }
    // Lane j: the score of the j-th choice, and the weights. Where they are divided
    // by their sum, a common factor is free: the softmax takes the largest chosen
    // logit as its reference, and scores of logits so small that fp32 would lose
    // them (sigmoid(z) = e^z, sqrt-softplus(z) = e^(z/2) there, to 1e-34) are
    // taken relative to the largest one's.
    const float zj = lane < a.k ? cleaned(row[e]) : -INFINITY;
    float s = 0.f;
    if (a.renorm) {
        const float zc = warp_max_value(zj);
        if (a.score_fn == MOE_SCORE_SOFTMAX)
            s = zc > -INFINITY ? expf(zj - zc) : 0.f;
        else if (zc < -80.f)
            s = zc > -INFINITY
                    ? expf(a.score_fn == MOE_SCORE_SIGMOID ? zj - zc : 0.5f * (zj - zc)) : 0.f;
        else
            s = score_value(zj, a.score_fn);
    } else {
        s = a.score_fn == MOE_SCORE_SOFTMAX ? expf(zj - zmax) : score_value(zj, a.score_fn);
    }
    float den = 1.f;
    if (a.renorm) {
        den = warp_sum(s);
    } else if (a.score_fn == MOE_SCORE_SOFTMAX) {
        float part = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q) part += expf(z[q] - zmax);  // 0 for an expert that is out
        den = warp_sum(part);
    }
    if (lane < a.k) {
        a.idx[t * a.k + lane] = e;
        a.w[t * a.k + lane] = den > 0.f ? a.scale * (s / den) : 0.f;
    }
}

}  // namespace

cudaError_t launch_select(const moe_config& c, const float* logits, long ld,
                          const float* score_bias, int score_fn, const moe_group_options& grp,
                          int32_t* idx, float* w, cudaStream_t s) {
    const SelectArgs a = {logits, ld, score_bias, score_fn, grp.n_group, grp.topk_group,
                          grp.group_score, grp.renormalize, c.T, c.E, c.k, c.scale, idx, w};
    const cudaError_t err = launch_pdl(select_kernel, dim3((unsigned)((c.T + WARPS - 1) / WARPS)),
                                       dim3(WARPS * 32), 0, s, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
