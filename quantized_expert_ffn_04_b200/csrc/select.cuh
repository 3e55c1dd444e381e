// Selection of tokens' experts by a routing rule, by the lanes of a warp (shared
// by strata_moe_route_logits and the layer's own routing).
//
// The rule (strata_moe.h, "Routing rules"): scores s by softmax or sigmoid,
// values v = s + b, groups of experts kept by their best value or the sum of
// their best two, the k largest values of the kept groups (a tie to the lower
// id), weights s over the picks.  Values are ordered as 64-bit arithmetic
// orders them.  That needs no 64-bit arithmetic for almost every token: the
// scores are computed in fp32 with a known error bound, and only where two
// values that decide something lie closer than the bound are they computed
// again in 64 bits.
//
// Bounds (the fp32 score of one expert against the real one, in units of 2^-24;
// ex2.approx is within 2^-22 relative, rcp.approx within 2^-23, and the rounded
// product l log2(e) moves the exponent by at most 1.5 |l|):
//   sigmoid  s (1 - s) (4 + 1.5 |l|) + 3 s <= 1 + 0.34 + 3, as s (1 - s) |l| <=
//            0.224 (3: the sum 1 + exp and the reciprocal);
//   softmax  p = exp(l - m) / Z, relative to the largest p, x = |l - m|: difference,
//            product, ex2 and the two roundings of 1 / Z give exp(-x) (6 + 2.5 x)
//            <= 6; Z sums its terms' relative errors, weighted by the terms,
//            4 + 2.5 * 7 (the mean of x under p is at most ln 1024 = 7), and NQ + 5
//            roundings (a lane's NQ terms, then the lanes).
// The sum v = s + b rounds by |v|.  The tolerances are twice the bounds (two
// values are compared), rounded up.
#pragma once

#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace strata {

constexpr float kSigmoidTol = 9 * 0x1p-24f;
constexpr float softmax_tol(int nq) { return (66 + 2 * nq) * 0x1p-24f; }
constexpr float kSumTol = 2.5f * 0x1p-24f;  // of |v|

// One token's logits.
struct LogitRow {
    const void *p;
    bool bf16;
    bool cg = false;  // written by this kernel's other blocks: read past L1
    // Logit e as the rule reads it: -inf for an expert that is not eligible (NaN
    // or -inf), +inf as the largest finite float.
    __device__ __forceinline__ float at(int e) const { return clean(raw(e)); }
    __device__ __forceinline__ float raw(int e) const {
        if (cg) return __ldcg(reinterpret_cast<const float *>(p) + e);
        return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[e])
                    : reinterpret_cast<const float *>(p)[e];
    }
    // the row that lane `src` works on
    __device__ __forceinline__ LogitRow of_lane(int src) const {
        return LogitRow{reinterpret_cast<const void *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), src)),
                        bf16, cg};
    }
    static __device__ __forceinline__ float clean(float l) {
        return l == l ? fminf(l, FLT_MAX) : -INFINITY;
    }
};

__device__ __forceinline__ bool before(double va, int ea, double vb, int eb) {
    return va > vb || (va == vb && ea < eb);
}
// Best two values: u joins (t1, t2).
template <typename V>
__device__ __forceinline__ void join_two(V u1, V u2, V &t1, V &t2) {
    const V lo = t1 < u1 ? t1 : u1;
    t1 = t1 > u1 ? t1 : u1;
    t2 = t2 > u2 ? t2 : u2;
    t2 = t2 > lo ? t2 : lo;
}

// ------------------------------------------------------------ 64-bit paths
// Reached by few tokens: out of line, reading the row again, so that the common
// path keeps its registers.

// Softmax: 1 / sum of exp(l - m) over all experts (sigmoid: unused).
static __device__ __noinline__ double inv_sum64(const SelectPlan &p, LogitRow row, int lane, float m) {
    if (p.score == STRATA_SCORE_SIGMOID) return 1.0;
    double z = 0.0;
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32) z += exp((double)row.at(e) - (double)m);
    for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return 1.0 / z;
}
static __device__ __noinline__ double score64(const SelectPlan &p, float l, float m, double inv_z) {
    if (p.score == STRATA_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-(double)l));
    return exp((double)l - (double)m) * inv_z;
}
// Ranking value; -inf for an expert that is not eligible.
__device__ __forceinline__ double value64(const SelectPlan &p, float l, int e, float m, double inv_z) {
    if (!p.bias || !(l > -INFINITY)) return (double)l;
    const double v = score64(p, l, m, inv_z) + (double)p.bias[e];
    return v == v ? v : -(double)INFINITY;
}

// The picks one after the other, from all experts of the kept groups: for
// tokens with more close candidates than lanes (many equal values) or with
// fewer eligible experts than picks.  Lane j gets pick j and its logit; the
// number of eligible picks is returned, later ones are the lowest other ids.
static __device__ __noinline__ int pick_rounds64(const SelectPlan &p, LogitRow row, int lane, float m, unsigned kept,
                                                 int &pick_e, float &pick_l) {
    const double none = -(double)INFINITY;
    const double inv_z = p.bias ? inv_sum64(p, row, lane, m) : 1.0;
    double last_v = (double)INFINITY;
    int last_e = -1, n = 0, found = 0;
    for (; n < p.k; n++) {
        double bv = none;
        int be = 0x7fffffff;
        for (int e = lane; e < p.E; e += 32) {
            double x = none;
            if ((kept >> (e / p.gs)) & 1) x = value64(p, row.at(e), e, m, inv_z);
            if (before(last_v, last_e, x, e) && before(x, e, bv, be)) {
                bv = x;
                be = e;
            }
        }
        for (int o = 16; o >= 1; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (before(ov, oe, bv, be)) {
                bv = ov;
                be = oe;
            }
        }
        if (lane == n) pick_e = be;
        found += bv > none;
        last_v = bv;
        last_e = be;
    }
    pick_l = lane < found ? row.at(pick_e) : 0.0f;
    return found;
}

// A pick's score for its weight, times a factor common to the token's picks:
// softmax exp(l - top) inv_z, sigmoid exp(-top) / (1 + exp(-l)) with top <= 0.
template <bool kSoftmax>
__device__ __forceinline__ float pick_score(float l, float top, float inv_z) {
    if (kSoftmax) return expf(l - top) * inv_z;
    return __fdividef(expf(fminf(l, 0.0f) - top), 1.0f + expf(-fabsf(l)));
}

// One token by the whole warp in 64 bits: picks and weights to idx and w.
static __device__ __noinline__ void slow_token(const SelectPlan &p, LogitRow row, int lane, float m, float inv_z,
                                               unsigned kept, int32_t *idx, float *w) {
    int e = 0;
    float l = 0.0f;
    const int n = pick_rounds64(p, row, lane, m, kept, e, l);
    float top = lane < n ? l : -INFINITY;
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s = 0.0f;
    if (lane < n) {
        if (p.score == STRATA_SCORE_SOFTMAX)
            s = p.renorm ? pick_score<true>(l, top, 1.0f) : pick_score<true>(l, m, inv_z);
        else
            s = pick_score<false>(l, p.renorm ? fminf(top, 0.0f) : 0.0f, 1.0f);
    }
    float sum = s;
    if (p.renorm) {
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s = sum > 0.0f ? s / sum : 0.0f;
    }
    if (lane < p.k) {
        idx[lane] = e;
        w[lane] = s * p.scale;
    }
}

// ------------------------------------------------------------ fast path
__device__ __forceinline__ float fast_exp(float x) {  // x <= 88: finite
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}
// score, and in `den` what is infinite where the logit may be -inf
template <bool kSoftmax>
__device__ __forceinline__ float fast_score(float l, float m, float inv_z, float &den) {
    if (kSoftmax) {
        den = l;
        return fast_exp(l - m) * inv_z;
    }
    float s;
    den = 1.0f + fast_exp(-l);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(den));
    return s;
}

// Reductions over the S lanes of a token (S a power of two).
template <int S>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = S / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int S, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
    for (int o = S / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Order-preserving integer of a float and back (no NaN).
__device__ __forceinline__ uint32_t ordered(float f) {
    const int u = __float_as_int(f);
    return (uint32_t)(u ^ ((u >> 31) | (int)0x80000000));
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// A token's close candidates, at most kCap of them, in the warp's shared memory:
// (value, expert) as one integer whose order is the rule's, value first, the
// lower expert on a tie.  0 is below all of them.
__device__ __forceinline__ unsigned long long candidate_key(float v, int e) {
    return ((unsigned long long)ordered(v + 0.0f) << 32) | (uint32_t)~e;  // -0 as +0
}
__device__ __forceinline__ float key_value(unsigned long long k) { return unordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_expert(unsigned long long k) { return (int)~(uint32_t)k; }

template <int S>
struct SelectScratch {
    static constexpr int kCap = S == 32 ? 64 : 32;
    unsigned long long c[32 / S][kCap];       // as found
    unsigned long long sorted[32 / S][kCap];  // by rank; the 64-bit path's values before that
};

// The lane layout: S lanes a token, L = 1 << ll of them a group; lane rl of
// group g holds the group's experts j = (i / 4) 4 L + 4 rl + i % 4 in element
// i < NQ.
struct SelectLanes {
    int step;     // 4 L
    int first;    // the lane's first expert
    int room;     // experts of the group from the lane's first one on (<= 0: none)
    bool padded;  // some lane's last elements are no experts
    __device__ __forceinline__ bool valid(int i) const { return (i >> 2) * step + (i & 3) < room; }
    __device__ __forceinline__ int expert(int i) const { return first + (i >> 2) * step + (i & 3); }
};

// Elements of an array (logits, biases): i .. i + 3, or all; 0 where there is no
// expert.  vec: four experts or none, aligned.
__device__ __forceinline__ void load_four(LogitRow row, bool vec, const SelectLanes &sl, int i, float (&f)[4]) {
    const int at = sl.first + (i >> 2) * sl.step;
    if (vec && !row.bf16) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 *q = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(row.p) + at);
        if (sl.valid(i)) u = row.cg ? __ldcg(q) : *q;
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
    } else if (vec) {
        uint2 u = make_uint2(0, 0);
        if (sl.valid(i)) u = *reinterpret_cast<const uint2 *>(reinterpret_cast<const __nv_bfloat16 *>(row.p) + at);
        f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
        f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int q = 0; q < 4; q++) f[q] = sl.valid(i + q) ? row.raw(at + q) : 0.0f;
    }
}
template <int NQ>
__device__ __forceinline__ void load_all(LogitRow row, bool vec, const SelectLanes &sl, float (&v)[NQ]) {
#pragma unroll
    for (int i = 0; i < NQ; i += 4) {
        float f[4];
        load_four(row, vec, sl, i, f);
#pragma unroll
        for (int q = 0; q < 4; q++) v[i + q] = f[q];
    }
}
template <int NQ>
__device__ __forceinline__ void load_elements(LogitRow row, bool vec, const SelectLanes &sl, float (&v)[NQ]) {
    // one branch round all the loads
    if (vec && !row.bf16) load_all<NQ>(LogitRow{row.p, false, row.cg}, true, sl, v);
    else if (vec) load_all<NQ>(LogitRow{row.p, true}, true, sl, v);
    else load_all<NQ>(row, false, sl, v);
}
template <int NQ>
__device__ __forceinline__ void mask_padding(const SelectLanes &sl, float (&v)[NQ]) {
    if (!sl.padded) return;
#pragma unroll
    for (int i = 0; i < NQ; i++) v[i] = sl.valid(i) ? v[i] : -INFINITY;
}
template <int S, int NQ>
__device__ __forceinline__ void softmax_stats(const float (&v)[NQ], float &m, float &inv_z) {
    float mx = v[0];
#pragma unroll
    for (int i = 1; i < NQ; i++) mx = fmaxf(mx, v[i]);
    mx = lanes_max<S>(mx);
    m = mx > -INFINITY ? mx : 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NQ; i++) z += fast_exp(v[i] - m);
    z = lanes_sum<S>(z);
    inv_z = z > 0.0f ? 1.0f / z : z;  // a NaN stays
}

// Logits v become ranking values (kBias: score + bias; else they stay); m and
// inv_z are set where softmax scores are needed.  kCareful: every logit is made
// the rule's first, and experts that are not eligible get -inf; without it,
// true is returned where that matters (a logit of -inf or NaN, a bias that is
// not finite).
template <int S, int NQ, bool kSoftmax, bool kBias, bool kCareful>
__device__ __forceinline__ bool rank_values(const SelectPlan &p, LogitRow row, bool vec, const SelectLanes &sl,
                                            const float4 *lane_bias, float (&v)[NQ], float &m, float &inv_z,
                                            bool scores) {
    float check = 0.0f;  // not finite where something is odd
    if (kCareful) {
        load_elements<NQ>(row, vec, sl, v);
#pragma unroll
        for (int i = 0; i < NQ; i++) v[i] = sl.valid(i) ? LogitRow::clean(v[i]) : -INFINITY;
    } else if (scores && (kSoftmax || !kBias)) {
#pragma unroll
        for (int i = 0; i < NQ; i++) check += v[i];
    }
    if (kSoftmax && (scores || !p.renorm)) {
        if (!kCareful) mask_padding<NQ>(sl, v);
        softmax_stats<S, NQ>(v, m, inv_z);
        check += inv_z;
    }
    if (kBias) {
#pragma unroll
        for (int i = 0; i < NQ; i += 4) {
            float b[4];
            if (S < 32) {
                const float4 u = lane_bias[(i >> 2) * S];
                b[0] = u.x, b[1] = u.y, b[2] = u.z, b[3] = u.w;
            } else {
                load_four(LogitRow{p.bias, false}, vec, sl, i, b);
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float den;
                const float x = fast_score<kSoftmax>(v[i + q], m, inv_z, den) + b[q];
                if (kCareful) {
                    v[i + q] = v[i + q] > -INFINITY && x == x ? x : -INFINITY;
                } else {
                    check = kSoftmax ? check + x : fmaf(den, x, check);
                    v[i + q] = x;
                }
            }
        }
    }
    if (!kCareful) mask_padding<NQ>(sl, v);
    return !(fabsf(check) < INFINITY);
}

// Softmax values x >= y with a bias that the tolerance of any two values could
// not tell apart: the bound of these two.  Z's error, most of the tolerance, is
// common to both scores, so only their difference carries it; the rest of a
// score's error is p (6 + 2.5 x) <= 6 p + 0.92 pmax.
template <int NQ>
__device__ __forceinline__ bool softmax_pair_close(float x, float y, float bx, float by, float pmax) {
    const float px = x - bx, py = y - by;
    const float units = 6.0f * (px + py) + 2.0f * pmax + (30.0f + NQ) * fabsf(px - py);
    return !(x - y > units * 0x1.1p-24f + 2.0f * kSumTol * fmaxf(fabsf(x), fmaxf(fabsf(bx), fabsf(by))));
}

// Softmax: 1 / sum in 64 bits of the lane's token, for the tokens with a bit in
// `which`.
template <int S, bool kSoftmax>
__device__ __forceinline__ double token_inv_sum64(const SelectPlan &p, LogitRow row, int lane, float m, unsigned which) {
    double iz = 1.0;
    if (kSoftmax)
        for (int s = 0; s < 32; s += S) {
            if (!((which >> s) & (S == 32 ? 0xffffffffu : (1u << (S & 31)) - 1u))) continue;
            const double x = inv_sum64(p, row.of_lane(s), lane, __shfl_sync(0xffffffffu, m, s));
            if (lane / S * S == s) iz = x;
        }
    return iz;
}

// Lane r of a token's S lanes.
template <int S>
__device__ __forceinline__ SelectLanes lanes_of(const SelectPlan &p, int r, int nq) {
    const int ll = (S == 32 ? 5 : S == 16 ? 4 : 3) - p.log2_groups, g = r >> ll, rl = r & ((1 << ll) - 1);
    const bool mine = g < p.n_groups;
    SelectLanes sl;
    sl.step = 4 << ll;
    sl.first = mine ? g * p.gs + 4 * rl : 0;
    sl.room = mine ? p.gs - 4 * rl : 0;
    sl.padded = (nq << ll) != p.gs || (1 << p.log2_groups) != p.n_groups;
    return sl;
}

// 32 / S tokens from t0 on by one warp; picks and weights of the tokens below T
// go to idx and w ([T][k]).  S < 32: `bias` is the selection bias in the lanes'
// order in shared memory, [NQ / 4][S] fours (read from global memory, a lane's
// experts lie in as many lines as there are lanes: 15 of 52 us at 65536 tokens
// of 256 experts).
template <int S, int NQ, bool kSoftmax, bool kBias>
__device__ __forceinline__ void select_tokens(const SelectPlan &p, const void *logits, bool bf16, bool vec,
                                              long long ld, int T, long long t0, const float4 *bias,
                                              SelectScratch<S> &scratch, int32_t *idx, float *w,
                                              bool cg = false) {
    constexpr int kCap = SelectScratch<S>::kCap, kOwn = kCap / S;
    constexpr bool kTwo = S < 32;  // the threshold from every lane's second best
    constexpr unsigned kAll = 0xffffffffu, kSub = S == 32 ? kAll : (1u << (S & 31)) - 1u;
    const int lane = threadIdx.x & 31, r = lane % S, base = lane - r;
    const long long t = t0 + lane / S < T ? t0 + lane / S : T - 1;
    const bool live = t0 + lane / S < T;
    const LogitRow row{reinterpret_cast<const char *>(logits) + t * ld * (bf16 ? 2 : 4), bf16, cg};
    const bool grouped = p.top_groups < p.n_groups;
    const bool group_scores = !kBias && grouped && p.sum2;
    const int ll = (S == 32 ? 5 : S == 16 ? 4 : 3) - p.log2_groups, g = r >> ll;
    const bool mine = g < p.n_groups;
    const SelectLanes sl = lanes_of<S>(p, r, NQ);

    float v[NQ], m = 0.0f, inv_z = 0.0f;
    load_elements<NQ>(row, vec, sl, v);
    const bool odd = rank_values<S, NQ, kSoftmax, kBias, false>(p, row, vec, sl, bias + r, v, m, inv_z, kBias || group_scores);
    if (__any_sync(kAll, odd))
        rank_values<S, NQ, kSoftmax, kBias, true>(p, row, vec, sl, bias + r, v, m, inv_z, kBias || group_scores);
    const float score_tol = kSoftmax ? softmax_tol(NQ) * inv_z : kSigmoidTol;

    // groups, and the lane's best (two) values
    float b1 = -INFINITY, b2 = -INFINITY;
    auto best_two = [&]() {
        b1 = b2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NQ; i += 2) {
            const float hi = fmaxf(v[i], v[i + 1]), lo = fminf(v[i], v[i + 1]);
            b2 = fmaxf(fmaxf(b2, lo), fminf(b1, hi));
            b1 = fmaxf(b1, hi);
        }
    };
    if (kTwo || grouped) {
        best_two();
    } else {
#pragma unroll
        for (int i = 0; i < NQ; i++) b1 = fmaxf(b1, v[i]);
    }
    bool kept = true;
    if (grouped) {
        float t1 = b1, t2 = b2;
        for (int o = 1; o < (1 << ll); o <<= 1)
            join_two(__shfl_xor_sync(kAll, t1, o), __shfl_xor_sync(kAll, t2, o), t1, t2);
        const bool two = p.sum2 && t2 > -INFINITY;
        float s1 = t1, s2 = t2, den;
        if (group_scores) {  // scores keep the logits' order
            s1 = t1 > -INFINITY ? fast_score<kSoftmax>(t1, m, inv_z, den) : -INFINITY;
            s2 = two ? fast_score<kSoftmax>(t2, m, inv_z, den) : -INFINITY;
        }
        // (without a bias a best value is the logit, +inf the largest finite float)
        const float gv = two ? s1 + s2 : kBias ? s1 : fminf(s1, FLT_MAX);
        // how many groups are ahead: a larger value, or the same and a lower id
        const uint32_t key = ordered(gv + 0.0f), lower = (1u << g) - 1u;
        int ahead = 0;
#pragma unroll 4
        for (int o = 0; o < p.n_groups; o++)
            ahead += __shfl_sync(kAll, key, o << ll, S) + ((lower >> o) & 1u) > key;
        kept = mine && ahead < p.top_groups;
        unsigned near64 = 0;
        if (kBias || p.sum2) {
            // the last group that stays and the first that goes: closer than any
            // two groups' bounds, and 64 bits decide
            const float size = gv > -INFINITY && mine ? fabsf(s1) + (two ? fabsf(s2) : 0.0f) : 0.0f;
            const float near = 2.0f * score_tol + 4.0f * kSumTol * lanes_max<S>(size);
            const int last = __ffs(__ballot_sync(kAll, mine && ahead == p.top_groups - 1) >> base & kSub) - 1;
            const int next = __ffs(__ballot_sync(kAll, mine && ahead == p.top_groups) >> base & kSub) - 1;
            const float low = __shfl_sync(kAll, gv, last, S), high = __shfl_sync(kAll, gv, next, S);
            near64 = __ballot_sync(kAll, high > -INFINITY && !(low - high > near));
        }
        if (near64) {
            const double none = -(double)INFINITY, iz = token_inv_sum64<S, kSoftmax>(p, row, lane, m, near64);
            double d1 = none, d2 = none;
            if (kBias) {
                // the few experts that may be the group's best (two)
                const float least = two ? t2 : t1;
                const float from = fabsf(least) < INFINITY ? least - (score_tol + kSumTol * fabsf(least)) : least;
                unsigned long long few = 0;
#pragma unroll
                for (int i = 0; i < NQ; i++) few |= (unsigned long long)(v[i] >= from && v[i] > -INFINITY) << i;
                for (; few; few &= few - 1) {
                    const int e = sl.expert(__ffsll((long long)few) - 1);
                    join_two(value64(p, row.at(e), e, m, iz), none, d1, d2);
                }
                for (int o = 1; o < (1 << ll); o <<= 1)
                    join_two(__shfl_xor_sync(kAll, d1, o), __shfl_xor_sync(kAll, d2, o), d1, d2);
            } else {
                if (t1 > -INFINITY) d1 = score64(p, t1, m, iz);
                if (two) d2 = score64(p, t2, m, iz);
            }
            const double gd = p.sum2 && d2 > none ? d1 + d2 : d1;
            ahead = 0;
            for (int o = 0; o < p.n_groups; o++) {
                const double other = __shfl_sync(kAll, gd, o << ll, S);
                ahead += other > gd || (other == gd && o < g);
            }
            if ((near64 >> base) & kSub) kept = mine && ahead < p.top_groups;
        }
        if (!kept) {
#pragma unroll
            for (int i = 0; i < NQ; i++) v[i] = -INFINITY;
            b1 = b2 = -INFINITY;
        }
    }

    // tau: a value that at least k experts reach.  Of the lanes' best, the k-th
    // largest; or, where the batch or the groups leave fewer lanes than picks, the
    // ceil(k / 2)-th largest of their second best, as each of those lanes holds two.
    // -inf when that is too few.
    const bool second = kTwo || (grouped && (p.top_groups << ll) < p.k);
    float tau = second ? b2 : b1;
#pragma unroll
    for (int size = 2; size <= S; size <<= 1)  // sorted over the lanes, largest first
#pragma unroll
        for (int o = size >> 1; o >= 1; o >>= 1) {
            const float x = __shfl_xor_sync(kAll, tau, o);
            tau = ((r & size) == 0) == ((r & o) == 0) ? fmaxf(tau, x) : fminf(tau, x);
        }
    tau = __shfl_sync(kAll, tau, second ? (p.k - 1) >> 1 : p.k - 1, S);
    const float tol = kBias ? score_tol : 0.0f, sum_tol = kBias ? kSumTol : 0.0f;
    auto reach = [&](float x) { return fabsf(x) < INFINITY ? x - (tol + sum_tol * fabsf(x)) : -FLT_MAX; };
    auto count = [&](float x) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < NQ; i++) n += v[i] >= x;
        return n;
    };
    // the place of the lane's candidates among the token's; their number
    auto place = [&](int cnt, int &total) {
        int end = cnt;
#pragma unroll
        for (int o = 1; o < S; o <<= 1) {
            const int x = __shfl_up_sync(kAll, end, o, S);
            if (r >= o) end += x;
        }
        total = __shfl_sync(kAll, end, S - 1, S);
        return end - cnt;
    };
    float thr = reach(tau);
    int total, pos = place(count(thr), total);
    // too many: bisect for a tau that between k and kCap experts reach
    if (__any_sync(kAll, total > kCap)) {
        uint32_t lo = ordered(thr), hi = ordered(lanes_max<S>(b1));
        bool done = total <= kCap || !(unordered(hi) < INFINITY);
        for (int step = 0; step < 32; step++) {
            if (hi - lo <= 1) done = true;
            if (__all_sync(kAll, done)) break;
            const uint32_t mid = lo + (hi - lo) / 2;
            const float x = unordered(mid);
            const int n = lanes_sum<S>(count(x));
            if (!done) {
                if (n < p.k) hi = mid;
                else if (n > kCap) lo = mid;
                else thr = reach(x), done = true;
            }
        }
        pos = place(count(thr), total);
    }
    const bool slow = total < p.k || total > kCap;

    if (!__all_sync(kAll, slow)) {
        unsigned long long *c = scratch.c[lane / S], *sorted = scratch.sorted[lane / S];
#pragma unroll
        for (int q = 0; q < kOwn; q++) c[r + q * S] = 0;
        __syncwarp();
        if (!slow) {
            float2 *at = reinterpret_cast<float2 *>(c) + pos;
#pragma unroll
            for (int i = 0; i < NQ; i++)
                if (v[i] >= thr) *at++ = make_float2(__int_as_float(sl.expert(i)), v[i]);
        }
        __syncwarp();
        const int n = slow ? 0 : total, most = (int)__reduce_max_sync(kAll, (unsigned)n);
#pragma unroll
        for (int q = 0; q < kOwn; q++) {
            if (q * S >= most) break;
            const float2 f = reinterpret_cast<const float2 *>(c)[r + q * S];
            // (without a bias a value is the logit, +inf the largest finite float)
            if (r + q * S < n) c[r + q * S] = candidate_key(kBias ? f.y : fminf(f.y, FLT_MAX), __float_as_int(f.x));
        }
        __syncwarp();
        // rank of candidates r, r + S, ...: how many are ahead
#pragma unroll
        for (int q = 0; q < kOwn; q++) {
            if (q * S >= most) break;
            const unsigned long long own = c[r + q * S];
            int ahead = 0;
            for (int j = 0; j < most; j += 4) {
#pragma unroll
                for (int u = 0; u < 4; u++) ahead += c[j + u] > own;
            }
            if (own) sorted[ahead] = own;
        }
        __syncwarp();
        if (kBias) {
            // neighbours closer than the bound: of the picks, and of the last pick with
            // those left out.  Softmax pairs have bounds of their own, which a value
            // further behind may exceed where the next one does not, so the last pick
            // is compared with every one that the common bound reaches.
            bool close = false;
            for (int a = r; a + 1 < n && (kSoftmax || a < p.k); a += S) {
                const unsigned long long kx = sorted[min(a, p.k - 1)], ky = sorted[a + 1];
                const float x = key_value(kx), y = key_value(ky);
                if (x - y > tol + sum_tol * fabsf(x)) continue;
                close = close || !kSoftmax || softmax_pair_close<NQ>(x, y, p.bias[key_expert(kx)], p.bias[key_expert(ky)], inv_z);
            }
            const unsigned near64 = __ballot_sync(kAll, close);
            if (near64) {
                const double iz = token_inv_sum64<S, kSoftmax>(p, row, lane, m, near64);
                const int n64 = ((near64 >> base) & kSub) ? n : 0;  // this token is one of them
                double *d = reinterpret_cast<double *>(sorted);
                double own[kOwn];
#pragma unroll
                for (int q = 0; q < kOwn; q++) {
                    const int a = r + q * S, e = a < n64 ? key_expert(c[a]) : 0;
                    own[q] = a < n64 ? value64(p, row.at(e), e, m, iz) : 0.0;
                    if (a < n64) d[a] = own[q];
                }
                __syncwarp();
                int rank[kOwn];
#pragma unroll
                for (int q = 0; q < kOwn; q++) {
                    const int a = r + q * S, e = a < n64 ? key_expert(c[a]) : 0;
                    rank[q] = 0;
                    for (int j = 0; a < n64 && j < n64; j++) rank[q] += before(d[j], key_expert(c[j]), own[q], e);
                }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < kOwn; q++)
                    if (r + q * S < n64) sorted[rank[q]] = c[r + q * S];
                __syncwarp();
            }
        }
        // picks r, r + S, ... and their weights, which are taken relative to the
        // largest pick where they sum to less than 2^-20 (for that token alone: a
        // token's weights do not depend on the warp's others), so that a score below
        // fp32's normal range belongs to a weight below 2^-106
        constexpr int kPicks = S < 32 ? 16 / S : 1;  // k <= 16 there
        float l[kPicks], s[kPicks], sum = 0.0f;
        int e[kPicks];
        const float top0 = kSoftmax ? (kBias ? m : n ? key_value(sorted[0]) : 0.0f) : 0.0f;
#pragma unroll
        for (int q = 0; q < kPicks; q++) {
            const int a = r + q * S;
            l[q] = s[q] = 0.0f;
            e[q] = 0;
            if (a < p.k && n) {
                e[q] = key_expert(sorted[a]);
                l[q] = kBias ? row.at(e[q]) : key_value(sorted[a]);
                s[q] = kSoftmax ? pick_score<kSoftmax>(l[q], p.renorm ? top0 : m, p.renorm ? 1.0f : inv_z)
                                : pick_score<kSoftmax>(l[q], 0.0f, 1.0f);
            }
            sum += s[q];
        }
        float f = 1.0f;
        if (p.renorm) {
            sum = lanes_sum<S>(sum);
            const bool tiny = sum < 0x1p-20f && n;
            if (__any_sync(kAll, tiny)) {
                float top = -INFINITY;
#pragma unroll
                for (int q = 0; q < kPicks; q++) top = r + q * S < p.k ? fmaxf(top, l[q]) : top;
                top = lanes_max<S>(top);
                if (!kSoftmax) top = fminf(top, 0.0f);
                sum = 0.0f;
#pragma unroll
                for (int q = 0; q < kPicks; q++) {
                    if (r + q * S < p.k && tiny) s[q] = pick_score<kSoftmax>(l[q], top, 1.0f);
                    sum += s[q];
                }
                sum = lanes_sum<S>(sum);
            }
            f = __fdividef(1.0f, sum);
        }
#pragma unroll
        for (int q = 0; q < kPicks; q++)
            if (r + q * S < p.k && n && live) {
                idx[t * p.k + r + q * S] = e[q];
                w[t * p.k + r + q * S] = s[q] * f * p.scale;  // scale / sum may leave fp32's range
            }
        __syncwarp();  // the scratch is free for the warp's next tokens
    }
    // one after the other: tokens with more equal values than the scratch holds
    // and tokens with fewer eligible experts than picks
    for (unsigned todo = __ballot_sync(kAll, slow && live && r == 0); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        const unsigned lanes = __ballot_sync(kAll, kept) >> src;
        unsigned stay = 0;
        for (int o = 0; o < p.n_groups; o++) stay |= ((lanes >> (o << ll)) & 1u) << o;
        const long long ts = t0 + src / S;
        slow_token(p, row.of_lane(src), lane, __shfl_sync(kAll, m, src), __shfl_sync(kAll, inv_z, src), stay, idx + ts * p.k,
                   w + ts * p.k);
    }
}

// ------------------------------------------------------------ kernel
// Warps of a block: more where they share the bias in shared memory.
template <int S>
constexpr int kSelectWarps = S == 32 ? 4 : 8;
// Blocks an SM holds at least (a bound on registers).  Batches: 64 registers
// (65536 tokens of 256 experts, 16 lanes each: 38.7 us, 52.6 without the bound;
// without groups and bias 20.6 and 26.0).  A token a warp: 72 (8192 tokens of 512:
// 8.8 us against 10.3); softmax values with a bias, which would spill there, 96
// (1037 tokens of 512: 4.6 us, 8.4 with 72 and 4.6 without a bound; 8192: 14.4,
// 14.8 and 13.7).
template <int S, int NQ, bool kSpills>
constexpr int kSelectBlocks = S < 32 ? 4 : NQ > 32 ? 2 : NQ > 16 ? 4 : kSpills ? 5 : 7;

template <int S, int NQ, bool kSoftmax, bool kBias>
__global__ __launch_bounds__(32 * kSelectWarps<S>, kSelectBlocks<S, NQ, kSoftmax && kBias>) void route_logits_kernel(
    const __grid_constant__ SelectPlan p, const void *__restrict__ logits, int bf16, int vec, long long ld,
    int T, int32_t *__restrict__ idx, float *__restrict__ w) {
    constexpr int kWarps = kSelectWarps<S>;
    __shared__ SelectScratch<S> scratch[kWarps];
    __shared__ float4 bias[S < 32 && kBias ? NQ / 4 * S : 1];
    grid_launch_dependents();
    grid_dependency_wait();
    if (S < 32 && kBias) {
        for (int f = threadIdx.x; f < NQ / 4 * S; f += 32 * kWarps) {
            float b[4];
            load_four(LogitRow{p.bias, false}, vec != 0, lanes_of<S>(p, f % S, NQ), f / S * 4, b);
            bias[f] = make_float4(b[0], b[1], b[2], b[3]);
        }
        __syncthreads();
    }
    const int warp = threadIdx.x >> 5;
    const long long t0 = ((long long)blockIdx.x * kWarps + warp) * (32 / S);
    if (t0 >= T) return;
    select_tokens<S, NQ, kSoftmax, kBias>(p, logits, bf16 != 0, vec != 0, ld, T, t0, bias, scratch[warp], idx, w);
}

// kBiased: instances for a selection bias too.
template <int S, int NQ, bool kBiased = true>
cudaError_t run_route(const SelectPlan &p, const void *logits, bool bf16, long long ld, int T,
                      int32_t *idx, float *w, bool vec, cudaStream_t s) {
    constexpr int kTokens = kSelectWarps<S> * (32 / S);  // a block
    const dim3 grid((unsigned)(((long long)T + kTokens - 1) / kTokens)), block(32 * kSelectWarps<S>);
    const bool softmax = p.score == STRATA_SCORE_SOFTMAX;
    auto *kernel = softmax ? route_logits_kernel<S, NQ, true, false> : route_logits_kernel<S, NQ, false, false>;
    if constexpr (kBiased)
        if (p.bias) kernel = softmax ? route_logits_kernel<S, NQ, true, true> : route_logits_kernel<S, NQ, false, true>;
    return launch_pdl(kernel, grid, block, 0, s, p, logits, bf16 ? 1 : 0, vec ? 1 : 0, ld, T, idx, w);
}

// Elements of a lane when S lanes take a token (rounded up to loads of four);
// too many when the lanes do not suffice for the groups.
inline int lane_elements(const SelectPlan &p, int S) {
    const int L = S >> p.log2_groups;
    return L ? 4 * ((p.gs + 4 * L - 1) / (4 * L)) : 1 << 20;
}

}  // namespace strata
