// select.cu -- the choice of experts from router logits: softmax, sigmoid or
// sqrt-softplus scores, a bias for the choice, groups of experts, top-k,
// weights with or without renormalisation.
//
//   s_e = score(z_e),  c_e = s_e (+ score_bias[e])
//   group score = max c, or the sum of the two largest c, of its experts
//   the topk_group best groups stay; the k largest c in them are chosen
//   w_j = scale * s_j (/ sum of the chosen s)
//
// One warp per token with up to 8 experts a lane (E <= 256). The scores increase
// with the logit, so without a bias the experts are ranked by the logits
// themselves; with one, and for sums of two scores, by fp32 evaluations. A token's
// common path is choose_packed on 32-bit keys. Where a comparison that decides
// something is closer than the bits cut off or the evaluation's error, the candidates
// are put in order by one fp64 evaluation a lane (order_exactly); where it is a group
// that is open, or the candidates themselves, the whole token is chosen once more with
// scores in fp64 (select_exactly, about 7 us for a token by itself). With a bias that
// is about one token in 500 together, without one in 50000, if the logits are fp32
// sums; logits of bf16 precision have equal values among the best nine of 256 in two
// tokens of five, which the order of the candidates settles: T = 16384 without a bias
// 13.0 us and 20.1, the softmax 13.4 and 20.6 (28.4 where it repeated whole tokens).
//
// Groups that do not fit a warp at 8 experts a lane, whole lanes and a power of two of
// them a group (E = 240 in 3, 5, 6 or 10 groups; more than 32 groups), take
// select_exactly for every token: T = 16384, E = 240 biased in 10 groups 66 us, in 8 27.
//
// Bound: instructions, about 600 a token without groups and 1000 with them, against
// 4 E bytes read. While its warps run, an SM issues in 70% of its cycles, its alu pipe
// is 56 to 60% busy, and a warp waits mostly for fixed latencies and its turn; the
// launch and the last tokens are the rest. Measured, E = 256, top-8, T = 16384, back
// to back: 13.0 us without a bias or groups (reading the logits takes 2.6); biased, E =
// 192 17.1 us; biased, 4 of 8 groups by their two best 25 to 29.5 us by the inputs, of
// which 4 and more are the latency of tokens with an open group. T = 64: 2.8 us, the
// launch's.
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int WARPS = 4;      // tokens per CTA
constexpr int Q = 8;          // experts per lane
constexpr int PAD_E = 256 + 8;
constexpr int kCtasPerSm = 7;  // persistent CTAs: 8 spill in the token loop, 6 leave issue slots

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

__device__ __forceinline__ uint32_t warp_max(uint32_t k) {
    return __reduce_max_sync(0xffffffffu, k);
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
    const uint32_t lo =
        __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((unsigned long long)hi << 32) | lo;
}
template <typename V>
__device__ __forceinline__ V warp_max_value(V v) { return value_of(warp_max(key_of(v))); }

__device__ __forceinline__ double warp_total(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The fp32 scores (softmax: before the division by the sum; z - max for z). The
// fast exponential is within |z| 2^-24 + 2^-22 of its value, which the sigmoid's
// slope s (1 - s) turns into at most 8e-8, the fast reciprocal adds 2 ulp, the sum
// with the bias half of one: together below 4e-7 of 1 + |c|, and the softmax's sum
// stays below that too. The sqrt-softplus is not bounded by 1: an error of 2e-7 of it
// remains where a bias cancels it, so that `unit`, 1 or a token's largest score to
// within 15%, takes the 1's place. The difference of two values is certain beyond
// kScoreError of unit + |c|.
constexpr float kScoreError = 1e-6f;
__device__ __forceinline__ float unit_of(int fn, float zmax) {
    return fn == MOE_SCORE_SQRT_SOFTPLUS ? sqrtf(fmaxf(zmax, 1.f)) : 1.f;
}
__device__ __forceinline__ float score_of(float z, int fn) {
    if (fn == MOE_SCORE_SOFTMAX) return __expf(z);
    if (fn == MOE_SCORE_SQRT_SOFTPLUS)
        return sqrtf(fmaxf(z, 0.f) + log1pf(__expf(-fabsf(z))));
    return __fdividef(1.0f, 1.0f + __expf(-z));
}
__device__ __forceinline__ double score_of(double z, int fn) {
    // the smallest scores, down to fp64's subnormals: e^z and e^(z/2) to 1e-17
    const bool root = fn == MOE_SCORE_SQRT_SOFTPLUS;
    if (z < -700.0) return exp(root ? 0.5 * z : z);
    if (root) return sqrt(fmax(z, 0.0) + log1p(exp(-fabs(z))));
    return 1.0 / (1.0 + exp(-z));
}

// How far a group's score, the largest value v1 (v2 = 0) or the sum v1 + v2,
// may be from its exact value: each term's error goes with its own magnitude, which
// the sum's may be far below (large biases of opposite signs). Two evaluations, 8e-7 unit +
// 4e-7 (|v1| + |v2|), and the sum's rounding and this bound's stay below it. A group
// without enough experts left has -infinity, exactly; sums that overflow stay open.
__device__ __forceinline__ float group_error(float unit, float v1, float v2) {
    return fminf(v1, v2) == -INFINITY ? 0.f : kScoreError * (unit + fabsf(v1) + fabsf(v2));
}

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

// One token's choice by one warp; lane j < k gets the j-th expert in `mine`. V
// float: no score takes part in a comparison; double: scores in 64 bits. (The
// score loop is rolled: this runs for single tokens, whose time is mostly that of
// fetching the instructions.)
template <typename V>
__device__ __forceinline__ void choose(const SelectArgs& a, const float (&z)[Q], float zmax,
                                       Scratch<V>& sc, int& mine) {
    using K = decltype(key_of(V()));
    const int lane = threadIdx.x & 31;
    const bool top2 = a.n_group > 1 && a.group_score == MOE_GROUP_TOP2;
    V r[Q], c[Q];  // what experts are ranked by; what groups sum
    if constexpr (sizeof(V) == 8) {
        V total = 1;
        if (a.score_fn == MOE_SCORE_SOFTMAX) {
            V part = 0;
#pragma unroll 1
            for (int q = 0; q < Q; ++q) part += exp((double)z[q] - (double)zmax);
            total = warp_total(part);  // (an expert that is out adds 0)
        }
#pragma unroll 1
        for (int q = 0; q < Q; ++q) {
            const int e = lane + 32 * q;
            V s = a.score_fn == MOE_SCORE_SOFTMAX ? exp((double)z[q] - (double)zmax) / total
                                                  : score_of((double)z[q], a.score_fn);
            if (a.bias && e < a.E) s += (V)cleaned(a.bias[e]);
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
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            int ahead = 0;
            const V own = sc.group[g < G ? g : 0];
            for (int o = 0; o < G; ++o) {
                const V v = sc.group[o];
                ahead += v > own || (v == own && o < g);
            }
            const uint32_t bits =
                __ballot_sync(0xffffffffu, g < G && ahead < a.topk_group);
            if (lane == 0) sc.kept[g0 >> 5] = bits;
        }
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

    for (int j = 0; j < a.k; ++j) {
        K best = key[0];
        int bq = 0;
#pragma unroll
        for (int q = 1; q < Q; ++q)
            if (key[q] > best) { best = key[q]; bq = q; }
        const K m = warp_max(best);
        const uint32_t e = __reduce_min_sync(0xffffffffu,
                                             best == m ? (uint32_t)(lane + 32 * bq) : 0xffffffffu);
        if (lane == j) mine = (int)e;
        if ((int)(e & 31u) == lane) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if ((int)(e >> 5) == q) key[q] = 0;
        }
    }
}

// The choice by one warp from its 8 values a lane, in one pass of 32-bit keys: the
// upper 29 bits of the value's order-preserving key, then 7 - q for the lane's
// q-th expert (of equal values the earlier one first). Each lane sorts its 8 keys
// once (19 compare-exchanges); a round is one redux.sync on the lanes' heads and a
// ballot. `mine`: 8 * lane + q of lane j's j-th expert, 0 <= j <= k (`exists`: there
// is one; lane k has the first that was left out). Values whose difference is
// within the cut-off bits or the evaluation's error (`error` and 1e-6 of them; 0:
// none was evaluated) leave their order open: kOrder
// if it is only that of these k + 1, kOpen if the k + 2nd may belong among them.
enum Certainty { kSure, kOrder, kOpen };
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}
__device__ __forceinline__ bool sure_order(uint32_t key, uint32_t next, float error) {
    if (error == 0.f || next == 0) return (key ^ next) > 7u;  // different after the cut
    const float v = key_value(key & ~7u), u = key_value(next & ~7u);
    const float big = fmaxf(fabsf(v), fabsf(u));
    return v - u > fmaf(1e-6f + kScoreError, big, error);  // (false for two -infinities)
}
__device__ __forceinline__ Certainty choose_packed(uint32_t (&h)[Q], int k, float error, int& mine,
                                                   bool& exists) {
    const int lane = threadIdx.x & 31;
    // a sorting network of 8 (Batcher's odd-even merge), descending
    exchange(h[0], h[1]); exchange(h[2], h[3]); exchange(h[4], h[5]); exchange(h[6], h[7]);
    exchange(h[0], h[2]); exchange(h[1], h[3]); exchange(h[4], h[6]); exchange(h[5], h[7]);
    exchange(h[1], h[2]); exchange(h[5], h[6]);
    exchange(h[0], h[4]); exchange(h[1], h[5]); exchange(h[2], h[6]); exchange(h[3], h[7]);
    exchange(h[2], h[4]); exchange(h[3], h[5]);
    exchange(h[1], h[2]); exchange(h[3], h[4]); exchange(h[5], h[6]);
    uint32_t key = 0, left_out = 0;  // lane j: the j-th key; the key after the last choice
    for (int j = 0; j <= k; ++j) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, h[0]);
        const int winner = __ffs(__ballot_sync(0xffffffffu, h[0] == m)) - 1;
        if (lane == j) {
            key = m;
            mine = winner * Q + 7 - (int)(m & 7u);
        }
        left_out = m;
        if (lane == winner) {
#pragma unroll
            for (int q = 0; q < Q - 1; ++q) h[q] = h[q + 1];
            h[Q - 1] = 0;
        }
    }
    // lane j: its choice against the next one (or the first one left out; 0: none is)
    uint32_t next = __shfl_down_sync(0xffffffffu, key, 1);
    if (lane == k - 1) next = left_out;
    exists = lane <= k && key != 0;
    if (__all_sync(0xffffffffu, lane >= k || sure_order(key, next, error))) return kSure;
    const uint32_t after = __reduce_max_sync(0xffffffffu, h[0]);
    const bool closed = left_out == 0 || after == 0 || sure_order(left_out, after, error);
    return closed && k < 32 ? kOrder : kOpen;
}

// The exact order of a token's k + 1 candidates (lane j: expert e, if `exists`), one
// evaluation in fp64 a lane: lane j gets the j-th. Not for a biased softmax, whose sum
// takes all experts. Out of line, as the whole token's repeat is.
__device__ __noinline__ int order_exactly(const SelectArgs& a, const float* row, int e,
                                          bool exists) {
    const int lane = threadIdx.x & 31;
    double v = -INFINITY;
    if (exists) {
        const float z = cleaned(row[e]);
        v = z;
        if (a.bias && z > -INFINITY) v = score_of(v, a.score_fn) + (double)cleaned(a.bias[e]);
    } else {
        e = 256;  // behind every expert
    }
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i <= a.k; ++i) {
        const double u = __shfl_sync(0xffffffffu, v, i);
        const int f = __shfl_sync(0xffffffffu, e, i);
        rank += u > v || (u == v && f < e);
    }
    int mine = 0;
#pragma unroll 1
    for (int i = 0; i <= a.k; ++i) {
        const int f = __shfl_sync(0xffffffffu, e, i);
        if (__shfl_sync(0xffffffffu, rank, i) == lane) mine = f;
    }
    return mine;
}

// A chosen expert's score in fp32, within 2 ulp of the exponential and 1 of the rest:
// sqrt-softplus(z) is e^(z/2) to 3e-8 below -16, which is a number long after e^z is none.
__device__ __forceinline__ float chosen_score(float z, int fn) {
    return fn == MOE_SCORE_SQRT_SOFTPLUS && z < -16.f ? expf(0.5f * z) : score_value(z, fn);
}

// Lane j < k: the weight of its expert from that expert's logit zj, in fp32 (4e-6 of the
// weight at most, which scales a bf16 output); z and zmax (the softmax's reference) are
// the token's. Where the weights are divided by their sum, a common factor is free: the
// softmax takes the largest chosen logit as its reference, and so do the others where
// that is below -20: sigmoid(z) = e^z and sqrt-softplus(z) = e^(z/2) there, to 2e-9, and
// the ratios to the largest stay numbers down to 1e-30. The difference of two logits
// is taken with its rounding's remainder.
__device__ __forceinline__ float weight_of(const SelectArgs& a, int fn, const float (&z)[Q],
                                           float zmax, float zj) {
    float s;
    if (a.renorm) {
        const float zc = warp_max_value(zj);
        if (fn == MOE_SCORE_SOFTMAX) {
            s = zc > -INFINITY ? expf(zj - zc) : 0.f;
        } else if (zc < -20.f) {
            const float d = zj - zc, v = d - zj, left = (zj - (d - v)) - (zc + v);
            const float half = fn == MOE_SCORE_SIGMOID ? 1.f : 0.5f, e = expf(half * d);
            s = zj > -INFINITY ? fmaf(e, half * left, e) : 0.f;
        } else {
            s = chosen_score(zj, fn);
        }
        const float den = warp_sum(s);
        return den > 0.f ? a.scale * __fdividef(s, den) : 0.f;
    }
    if (fn != MOE_SCORE_SOFTMAX) return a.scale * chosen_score(zj, fn);
    float part = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) part += expf(z[q] - zmax);  // 0 for an expert that is out
    const float den = warp_sum(part);
    return den > 0.f ? a.scale * (expf(zj - zmax) / den) : 0.f;
}

__device__ __forceinline__ float largest(const float (&z)[Q]) {
    float m = z[0];
#pragma unroll
    for (int q = 1; q < Q; ++q) m = fmaxf(m, z[q]);
    m = warp_max_value(m);
    return m == -INFINITY ? 0.f : m;  // every expert is out: all scores 0
}

// A token's choice and weights without a cut: logits as they are, scores in fp64.
// Out of line: the common path keeps its registers.
__device__ __noinline__ void select_exactly(const SelectArgs& a, long t, WarpScratch& scratch) {
    const int lane = threadIdx.x & 31;
    const float* row = a.logits + t * a.ld;
    float z[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        z[q] = lane + 32 * q < a.E ? cleaned(row[lane + 32 * q]) : -INFINITY;
    const float zmax = a.score_fn == MOE_SCORE_SOFTMAX ? largest(z) : 0.f;
    int e = 0;
    __syncwarp();
    if (a.bias || (a.n_group > 1 && a.group_score == MOE_GROUP_TOP2))
        choose<double>(a, z, zmax, scratch.d, e);
    else
        choose<float>(a, z, zmax, scratch.f, e);
    __syncwarp();
    const float w = weight_of(a, a.score_fn, z, zmax, lane < a.k ? cleaned(row[e]) : -INFINITY);
    if (lane < a.k) {
        a.idx[t * a.k + lane] = e;
        a.w[t * a.k + lane] = w;
    }
}

// Persistent warps, a token each in turn, the next token's logits on the way. The
// packed choice is tried first; the tokens it leaves open (a bit each, of up to
// 64) follow exactly. GROUPS: `lanes` (a power of two) lanes hold one group of n
// experts, 8 a lane, so that a group's score is a few shuffles; otherwise lane l
// holds the experts l, l + 32, ...
template <int FN, bool GROUPS>
__global__ void __launch_bounds__(WARPS * 32, kCtasPerSm)
select_kernel(const __grid_constant__ SelectArgs a, int lanes) {
    pdl_launch_and_wait();
    __shared__ WarpScratch scratch[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = a.E / a.n_group;  // experts of a group
    const int shift = __ffs(lanes) - 1;
    const int group = lane >> shift, sub = lane & (lanes - 1);
    auto expert = [&](int q) { return GROUPS ? group * n + sub * Q + q : lane + 32 * q; };
    auto exists = [&](int q) {
        return GROUPS ? group < a.n_group && sub * Q + q < n : lane + 32 * q < a.E;
    };
    const bool top2 = GROUPS && a.group_score == MOE_GROUP_TOP2;
    const bool evaluated = a.bias || top2;  // scores take part in a comparison
    float bias[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) bias[q] = a.bias && exists(q) ? cleaned(a.bias[expert(q)]) : 0.f;
    const long step = (long)gridDim.x * WARPS;
    float coming[Q];  // the next token's logits
    auto load = [&](long t) {
        const float* p = a.logits + t * a.ld + (GROUPS ? group * n + sub * Q : lane);
#pragma unroll
        for (int q = 0; q < Q; ++q) coming[q] = exists(q) ? p[GROUPS ? q : 32 * q] : -INFINITY;
    };
    long t = (long)blockIdx.x * WARPS + warp;
    if (t < a.T) load(t);
    while (t < a.T) {
        const long t0 = t;
        unsigned long long open = 0;
        for (int i = 0; i < 64 && t < a.T; ++i, t += step) {
            float z[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) z[q] = cleaned(coming[q]);
            if (t + step < a.T) load(t + step);
            const float zmax = FN == MOE_SCORE_SOFTMAX ||
                                       (FN == MOE_SCORE_SQRT_SOFTPLUS && evaluated)
                                   ? largest(z) : 0.f;
            const float unit = unit_of(FN, zmax);
            // what experts are ranked by, and what groups sum
            float c[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) c[q] = z[q];
            if (evaluated) {
                float inv = 1.f;
                if (FN == MOE_SCORE_SOFTMAX) {
                    float part = 0.f;
#pragma unroll
                    for (int q = 0; q < Q; ++q) part += __expf(z[q] - zmax);
                    inv = __fdividef(1.f, warp_sum(part));
                }
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float s = FN == MOE_SCORE_SOFTMAX ? __expf(z[q] - zmax) * inv
                                                            : score_of(z[q], FN);
                    c[q] = z[q] == -INFINITY ? -INFINITY : s + bias[q];
                }
            }
            bool sure = true, kept = true;
            if (GROUPS) {
                float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    v2 = fmaxf(v2, fminf(v1, c[q]));
                    v1 = fmaxf(v1, c[q]);
                }
                for (int o = 1; o < lanes; o <<= 1) {
                    const float u1 = __shfl_xor_sync(0xffffffffu, v1, o);
                    const float u2 = __shfl_xor_sync(0xffffffffu, v2, o);
                    v2 = fmaxf(fmaxf(v2, u2), fminf(v1, u1));
                    v1 = fmaxf(v1, u1);
                }
                const float own = top2 ? v1 + v2 : v1;
                int ahead = 0;  // a group stays if fewer than topk_group are ahead of it
                for (int g = 0; g < a.n_group; ++g) {
                    const float v = __shfl_sync(0xffffffffu, own, g << shift);
                    ahead += v > own || (v == own && g < group);
                }
                kept = ahead < a.topk_group;
                if (evaluated && a.topk_group < a.n_group) {
                    // the least a kept group may be worth against the most another may
                    // (two -infinities: the index decides)
                    const bool is = group < a.n_group;
                    const float error = group_error(unit, v1, top2 ? v2 : 0.f);
                    const float least = own == -INFINITY ? own : fmaxf(own - error, -FLT_MAX);
                    const float low = key_value(
                        __reduce_min_sync(0xffffffffu, kept && is ? order_key(least) : ~0u));
                    const uint32_t high =
                        __reduce_max_sync(0xffffffffu, kept || !is ? 0u : order_key(own + error));
                    sure = key_value(high) == -INFINITY || low > key_value(high);
                }
            }
            uint32_t h[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q)
                h[q] = kept && exists(q)
                           ? (order_key(top2 && !a.bias ? z[q] : c[q]) & ~7u) | (uint32_t)(7 - q)
                           : 0u;
            int e = 0;
            bool candidate;
            const Certainty order =
                choose_packed(h, a.k, a.bias ? kScoreError * unit : 0.f, e, candidate);
            if (!sure || order == kOpen ||
                (order == kOrder && FN == MOE_SCORE_SOFTMAX && a.bias)) {
                open |= 1ull << i;
                continue;
            }
            const int l = e >> 3, q = e & 7;
            e = GROUPS ? (l >> shift) * n + (l & (lanes - 1)) * Q + q : l + 32 * q;
            const float* row = a.logits + t * a.ld;
            if (order == kOrder) e = order_exactly(a, row, e, candidate);
            const float w =
                weight_of(a, FN, z, zmax, lane < a.k ? cleaned(row[e]) : -INFINITY);
            if (lane < a.k) {
                a.idx[t * a.k + lane] = e;
                a.w[t * a.k + lane] = w;
            }
        }
        while (open) {
            const int i = __ffsll((long long)open) - 1;
            open &= open - 1;
            select_exactly(a, t0 + i * step, scratch[warp]);
        }
    }
}

// Groups that do not fit a warp's lanes (more than 32 / lanes of them): every token in
// fp64 where scores are compared, the measured cost of which the header gives.
__global__ void __launch_bounds__(WARPS * 32, kCtasPerSm)
select_exact_kernel(const __grid_constant__ SelectArgs a) {
    pdl_launch_and_wait();
    __shared__ WarpScratch scratch[WARPS];
    const int warp = threadIdx.x >> 5;
    for (long t = (long)blockIdx.x * WARPS + warp; t < a.T; t += (long)gridDim.x * WARPS)
        select_exactly(a, t, scratch[warp]);
}

template <int FN>
cudaError_t launch(const SelectArgs& a, cudaStream_t s) {
    const long ctas = ((long)a.T + WARPS - 1) / WARPS, most = 148L * kCtasPerSm;
    const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(WARPS * 32);
    if (a.n_group == 1) return launch_pdl(select_kernel<FN, false>, grid, block, 0, s, a, 1);
    int lanes = 1;
    while (lanes * Q < a.E / a.n_group) lanes *= 2;
    if (lanes * a.n_group <= 32)
        return launch_pdl(select_kernel<FN, true>, grid, block, 0, s, a, lanes);
    return launch_pdl(select_exact_kernel, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_select(const moe_config& c, const float* logits, long ld,
                          const float* score_bias, int score_fn, const moe_group_options& grp,
                          int32_t* idx, float* w, cudaStream_t s) {
    const SelectArgs a = {logits, ld, score_bias, score_fn, grp.n_group, grp.topk_group,
                          grp.group_score, grp.renormalize, c.T, c.E, c.k, c.scale, idx, w};
    const cudaError_t err = score_fn == MOE_SCORE_SOFTMAX ? launch<MOE_SCORE_SOFTMAX>(a, s)
                            : score_fn == MOE_SCORE_SQRT_SOFTPLUS
                                ? launch<MOE_SCORE_SQRT_SOFTPLUS>(a, s)
                                : launch<MOE_SCORE_SIGMOID>(a, s);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
