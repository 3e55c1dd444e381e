// Warp-level selection of one token's experts by a routing rule (shared by
// strata_moe_route_logits and the layer's own routing).
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
// Bounds (the fp32 score of one expert against the real one; CUDA documents
// __expf(x) within (2 + 1.173 |x|) ulp and __fdividef within 2 ulp, an ulp being
// at most 2^-23 relative):
//   sigmoid  s (1 - s) (2 + 1.173 |l|) 2^-23 + s (2 2^-23 + 2^-24)
//            <= (0.5 + 0.263 + 2.5) 2^-23 = 3.9e-7, as s (1 - s) |l| <= 0.224;
//   softmax  p = exp(l - m) / Z, relative to the largest p: the difference's
//            rounding and __expf give at most (2 + 0.63) 2^-23 (x exp(-x) <= 0.37);
//            Z sums up to 64 + 5 roundings of 2^-24 and its terms' own relative
//            errors, weighted by the terms: (2 + 1.7 * 7) 2^-23 when the mean
//            of |l - m| under p is at most ln 1024 = 7; together <= 6.2e-6.
// The sum v = s + b rounds by 2^-24 |v|.  kSigmoidTol and kSoftmaxTol are twice
// the bounds (two values are compared), padded.
#pragma once

#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace strata {

constexpr float kSigmoidTol = 1e-6f;
constexpr float kSoftmaxTol = 1.4e-5f;
constexpr float kSumTol = 1.5e-7f;  // of |v|: two roundings of 2^-24, padded

// A candidate of one token's top-k.
struct SelectSlot {
    float v;
    int e;
};

// One token's logits.
struct LogitRow {
    const void *p;
    bool bf16;
    // Logit e as the rule reads it: -inf for an expert that is not eligible (NaN
    // or -inf), +inf as the largest finite float.
    __device__ __forceinline__ float at(int e) const {
        const float l = bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[e])
                             : reinterpret_cast<const float *>(p)[e];
        return clean(l);
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
    if (!p.bias) return (double)l;
    const double v = score64(p, l, m, inv_z) + (double)p.bias[e];
    return l > -INFINITY && v == v ? v : -(double)INFINITY;
}

// The groups that stay, as a bit mask.
static __device__ __noinline__ unsigned keep_groups64(const SelectPlan &p, LogitRow row, int lane, float m) {
    const double none = -(double)INFINITY;
    const double inv_z = inv_sum64(p, row, lane, m);
    double mine = none;  // lane g: group g's value
    for (int g = 0; g < p.n_groups; g++) {
        double t1 = none, t2 = none;
        for (int j = lane; j < p.gs; j += 32) {
            const int e = g * p.gs + j;
            const float l = row.at(e);
            double x = value64(p, l, e, m, inv_z);
            if (p.sum2 && !p.bias && l > -INFINITY) x = score64(p, l, m, inv_z);
            join_two(x, none, t1, t2);
        }
        for (int o = 16; o >= 1; o >>= 1)
            join_two(__shfl_xor_sync(0xffffffffu, t1, o), __shfl_xor_sync(0xffffffffu, t2, o), t1, t2);
        if (lane == g) mine = p.sum2 && t2 > none ? t1 + t2 : t1;
    }
    int rank = 0;
    for (int o = 0; o < p.n_groups; o++) {
        const double other = __shfl_sync(0xffffffffu, mine, o);
        rank += other > mine || (other == mine && o < lane);
    }
    return __ballot_sync(0xffffffffu, lane < p.n_groups && rank < p.top_groups);
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

// ------------------------------------------------------------ one token
// fp32 score of a logit.
__device__ __forceinline__ float fast_score(bool softmax, float l, float m, float inv_z) {
    return softmax ? __expf(l - m) * inv_z : __fdividef(1.0f, 1.0f + __expf(-l));
}

// One token by one warp.  Lane group g = lane / L holds expert group g (L =
// 1 << log2_lanes); lane r of it holds the group's experts
// j = (i / 4) 4 L + 4 r + i % 4 in v[i], i < NQ: the rule's logits (-inf where
// there is no expert), which become ranking values.  bias[i] likewise.
// `slots`: 32 entries of the warp's shared memory.  A lane whose `rank` ends
// below k holds that pick and its weight.
template <int NQ>
__device__ __forceinline__ void select_token(const SelectPlan &p, LogitRow row, int lane, float (&v)[NQ],
                                             const float (&bias)[NQ], SelectSlot *slots, int &rank, int &pick_e,
                                             float &pick_w) {
    const bool softmax = p.score == STRATA_SCORE_SOFTMAX;
    const bool biased = p.bias != nullptr;
    const bool grouped = p.top_groups < p.n_groups;
    const int g = lane >> p.log2_lanes;
    float m = 0.0f, inv_z = 0.0f;
    if (softmax && (biased || (p.sum2 && grouped) || !p.renorm)) {
        float mx = v[0];
#pragma unroll
        for (int i = 1; i < NQ; i++) mx = fmaxf(mx, v[i]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        m = mx > -INFINITY ? mx : 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < NQ; i++) z += __expf(v[i] - m);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        inv_z = z > 0.0f ? 1.0f / z : 0.0f;
    }
    if (biased) {
#pragma unroll
        for (int i = 0; i < NQ; i++) {
            const float x = fast_score(softmax, v[i], m, inv_z) + bias[i];
            v[i] = v[i] > -INFINITY && x == x ? x : -INFINITY;
        }
    }
    const float score_tol = softmax ? kSoftmaxTol * inv_z : kSigmoidTol;

    unsigned kept_mask = 0xffffffffu;
    if (grouped) {
        float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NQ; i++) {
            float x = v[i];
            if (p.sum2 && !biased) x = x > -INFINITY ? fast_score(softmax, x, m, inv_z) : x;
            t2 = fmaxf(t2, fminf(t1, x));
            t1 = fmaxf(t1, x);
        }
        for (int o = 1; o < (1 << p.log2_lanes); o <<= 1)
            join_two(__shfl_xor_sync(0xffffffffu, t1, o), __shfl_xor_sync(0xffffffffu, t2, o), t1, t2);
        const bool two = p.sum2 && t2 > -INFINITY;
        const float gv = two ? t1 + t2 : t1;
        int ahead = 0;
        for (int o = 0; o < p.n_groups; o++) {
            const float other = __shfl_sync(0xffffffffu, gv, o << p.log2_lanes);
            ahead += other > gv || (other == gv && o < g);
        }
        bool kept = g < p.n_groups && ahead < p.top_groups;
        if (biased || p.sum2) {
            // the smallest value that stays and the largest that goes, and the
            // largest magnitude that went into a sum
            float low = kept ? gv : INFINITY, high = kept ? -INFINITY : gv;
            float mag = t1 > -INFINITY ? fabsf(t1) + (two ? fabsf(t2) : 0.0f) : 0.0f;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
                high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
                mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, o));
            }
            if (high > -INFINITY && !(low - high > 2.0f * score_tol + 3.0f * kSumTol * mag)) {
                const unsigned by_group = keep_groups64(p, row, lane, m);
                kept = g < p.n_groups && ((by_group >> g) & 1);
            }
        }
        kept_mask = 0;
        const unsigned by_lane = __ballot_sync(0xffffffffu, kept);
        for (int o = 0; o < p.n_groups; o++) kept_mask |= ((by_lane >> (o << p.log2_lanes)) & 1u) << o;
#pragma unroll
        for (int i = 0; i < NQ; i++) v[i] = kept ? v[i] : -INFINITY;
    }

    // tau: at least k experts reach it, the k-th largest of the lanes' own best
    // (32 values sorted over the lanes, largest first)
    float best = v[0];
#pragma unroll
    for (int i = 1; i < NQ; i++) best = fmaxf(best, v[i]);
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o >= 1; o >>= 1) {
            const float x = __shfl_xor_sync(0xffffffffu, best, o);
            const bool take_max = ((lane & size) == 0) == ((lane & o) == 0);
            best = take_max ? fmaxf(best, x) : fminf(best, x);
        }
    const float tau = __shfl_sync(0xffffffffu, best, p.k - 1);
    const float tol = biased ? score_tol : 0.0f;
    const float sum_tol = biased ? kSumTol : 0.0f;
    const float thr = fabsf(tau) < INFINITY ? tau - (tol + sum_tol * fabsf(tau)) : -FLT_MAX;
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < NQ; i++) cnt += v[i] >= thr;
    int pos = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, pos, o);
        if (lane >= o) pos += x;
    }
    const int total = __shfl_sync(0xffffffffu, pos, 31);
    pos -= cnt;
    float pl;       // the pick's logit
    int n = p.k;    // picks that are eligible
    if (total >= p.k && total <= 32) {
#pragma unroll
        for (int i = 0; i < NQ; i++)
            if (v[i] >= thr) {
                slots[pos].v = v[i];
                slots[pos].e = g * p.gs + ((i >> 2) << (p.log2_lanes + 2)) +
                               4 * (lane & ((1 << p.log2_lanes) - 1)) + (i & 3);
                pos++;
            }
        __syncwarp();
        const bool have = lane < total;
        const SelectSlot c = slots[have ? lane : 0];
        pl = row.at(c.e);
        rank = 0;
        bool close = false;
        const float mine = tol + sum_tol * fabsf(c.v);
        for (int j = 0; j < total; j++) {
            const SelectSlot o = slots[j];
            rank += o.v > c.v || (o.v == c.v && o.e < c.e);
            close |= o.e != c.e && !(fabsf(o.v - c.v) > mine);
        }
        if (biased && __any_sync(0xffffffffu, close)) {
            const double cd = value64(p, pl, c.e, m, inv_sum64(p, row, lane, m));
            rank = 0;
            for (int j = 0; j < total; j++) {
                const double od = __shfl_sync(0xffffffffu, cd, j);
                const int oe = __shfl_sync(0xffffffffu, c.e, j);
                rank += before(od, oe, cd, c.e);
            }
        }
        if (!have) rank = 32;
        pick_e = c.e;
        __syncwarp();  // the slots are free for the warp's next token
    } else {
        n = pick_rounds64(p, row, lane, m, kept_mask, pick_e, pl);
        rank = lane;
    }
    // Weights from the picks' logits.  Renormalised ones are taken relative to
    // the largest pick, so that picks with tiny scores keep their ratios.
    const bool mine = rank < n;
    float top = mine ? pl : -INFINITY;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s;
    if (softmax) {
        s = p.renorm ? expf(pl - top) : expf(pl - m) * inv_z;
    } else {
        const float c = p.renorm ? fminf(top, 0.0f) : 0.0f;
        s = pl > 0.0f ? 1.0f / (1.0f + expf(-pl)) : expf(pl - c) / (1.0f + expf(pl));
    }
    s = mine ? s : 0.0f;
    if (p.renorm) {
        float sum = s;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s = sum > 0.0f ? s / sum : 0.0f;
    }
    pick_w = s * p.scale;
}

}  // namespace strata
