// Routing rules: picks and weights from logits (strata_moe_route_logits), and
// the same kernel for a layer whose rule is set (strata_moe_set_routing).
//
// One warp per token (select.cuh).  The work is one read of the logits and a
// few hundred instructions a token.
#include <math.h>
#include <stdio.h>

#include "common.cuh"
#include "internal.h"
#include "select.cuh"

namespace strata {

constexpr int kSelectWarps = 4;

// Four logits (or biases) of a lane: experts j .. j + 3 of a group of gs, e0
// the group's first.  Entries past the group are -inf.
template <bool kVec>
__device__ __forceinline__ void load_four(LogitRow row, int e0, int j, int gs, float (&out)[4]) {
    float f[4];
    if (kVec) {  // gs a multiple of 4 and the row aligned: all four or none
        const int e = e0 + (j < gs ? j : 0);
        if (row.bf16) {
            const uint2 u = *reinterpret_cast<const uint2 *>(reinterpret_cast<const __nv_bfloat16 *>(row.p) + e);
            f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
            f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
        } else {
            const float4 u = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(row.p) + e);
            f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
        }
#pragma unroll
        for (int q = 0; q < 4; q++) out[q] = j < gs ? LogitRow::clean(f[q]) : -INFINITY;
    } else {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float l = row.at(e0 + (j + q < gs ? j + q : 0));
            out[q] = j + q < gs ? l : -INFINITY;
        }
    }
}

template <int NQ, bool kVec>
__global__ __launch_bounds__(32 * kSelectWarps) void route_logits_kernel(
    const __grid_constant__ SelectPlan p, const void *__restrict__ logits, int bf16, long long ld,
    int T, int32_t *__restrict__ idx, float *__restrict__ w) {
    __shared__ SelectSlot slots[kSelectWarps][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * kSelectWarps + warp;
    if (t >= T) return;
    const int L = 1 << p.log2_lanes, g = lane >> p.log2_lanes, r = lane & (L - 1);
    const bool active = g < p.n_groups;
    const int e0 = active ? g * p.gs : 0, gs = active ? p.gs : 0;
    const LogitRow row{reinterpret_cast<const char *>(logits) + (long long)t * ld * (bf16 ? 2 : 4), bf16 != 0};
    const LogitRow brow{p.bias, false};
    float v[NQ], b[NQ];
#pragma unroll
    for (int i = 0; i < NQ; i += 4) {
        float f[4];
        const int j = i * L + 4 * r;
        load_four<kVec>(row, e0, j, gs, f);
#pragma unroll
        for (int q = 0; q < 4; q++) v[i + q] = f[q];
        if (p.bias) load_four<false>(brow, e0, j, gs, f);
#pragma unroll
        for (int q = 0; q < 4; q++) b[i + q] = p.bias ? f[q] : 0.0f;
    }
    int rank, e;
    float wt;
    select_token<NQ>(p, row, lane, v, b, slots[warp], rank, e, wt);
    if (rank < p.k) {
        idx[(long long)t * p.k + rank] = e;
        w[(long long)t * p.k + rank] = wt;
    }
}

template <int NQ>
static cudaError_t run_route(const SelectPlan &p, const void *logits, bool bf16, long long ld, int T,
                             int32_t *idx, float *w, bool vec, cudaStream_t s) {
    const dim3 grid((T + kSelectWarps - 1) / kSelectWarps), block(32 * kSelectWarps);
    return launch_pdl(vec ? route_logits_kernel<NQ, true> : route_logits_kernel<NQ, false>, grid,
                      block, 0, s, p, logits, bf16 ? 1 : 0, ld, T, idx, w);
}

cudaError_t launch_route_logits(const SelectPlan &p, const void *logits, bool bf16, long long ld,
                                int T, int32_t *idx, float *w, cudaStream_t s) {
    // four logits a load where every group of every row starts at a multiple of it
    const bool vec = p.gs % 4 == 0 && ld % 4 == 0 && ((uintptr_t)logits % (bf16 ? 8 : 16)) == 0;
    const int L = 1 << p.log2_lanes, nq = 4 * ((p.gs + 4 * L - 1) / (4 * L));
    if (nq <= 4) return run_route<4>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (nq <= 8) return run_route<8>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (nq <= 16) return run_route<16>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (nq <= 32) return run_route<32>(p, logits, bf16, ld, T, idx, w, vec, s);
    return run_route<64>(p, logits, bf16, ld, T, idx, w, vec, s);  // 1024 / 17 = 60 experts a lane
}

strata_status make_select_plan(const strata_moe_routing *rule, int E, int k, const char *who,
                               SelectPlan *plan) {
    char buf[256];
    const char *what = nullptr;
    if (!rule)
        what = "rule is NULL";
    else if (rule->score != STRATA_SCORE_SOFTMAX && rule->score != STRATA_SCORE_SIGMOID)
        what = "score must be STRATA_SCORE_SOFTMAX or STRATA_SCORE_SIGMOID";
    else if (rule->group_score != STRATA_GROUP_BEST && rule->group_score != STRATA_GROUP_SUM2)
        what = "group_score must be STRATA_GROUP_BEST or STRATA_GROUP_SUM2";
    else if (rule->renorm != 0 && rule->renorm != 1)
        what = "renorm must be 0 or 1";
    else if (!std::isfinite(rule->scale))
        what = "scale must be finite";
    else if (rule->n_groups < 1 || rule->n_groups > 32 || E % rule->n_groups != 0)
        what = "n_groups must be 1..32 and divide the number of experts";
    else if (rule->top_groups < 1 || rule->top_groups > rule->n_groups)
        what = "top_groups must be 1..n_groups";
    else if (k > rule->top_groups * (E / rule->n_groups))
        what = "top_groups groups hold fewer than k experts";
    else if (rule->group_score == STRATA_GROUP_SUM2 && E / rule->n_groups < 2)
        what = "STRATA_GROUP_SUM2 needs groups of at least two experts";
    if (what) {
        snprintf(buf, sizeof buf, "%s: %s", who, what);
        set_error_message(buf);
        return STRATA_ERR_INVALID_ARG;
    }
    SelectPlan p{};
    p.E = E;
    p.k = k;
    p.score = rule->score;
    p.renorm = rule->renorm;
    // groups of which all stay leave nothing out
    const bool grouped = rule->top_groups < rule->n_groups;
    p.n_groups = grouped ? rule->n_groups : 1;
    p.top_groups = grouped ? rule->top_groups : 1;
    p.gs = E / p.n_groups;
    p.sum2 = grouped && rule->group_score == STRATA_GROUP_SUM2;
    p.log2_lanes = 5;
    while ((32 >> p.log2_lanes) < p.n_groups) p.log2_lanes--;
    p.scale = rule->scale;
    *plan = p;
    return STRATA_OK;
}

}  // namespace strata

using namespace strata;

extern "C" strata_status strata_moe_route_logits(const strata_moe_routing *rule,
                                                 const void *logits_dev, int logits_type,
                                                 int64_t ld, const float *select_bias_dev, int T,
                                                 int E, int k, int32_t *idx_dev, float *w_dev,
                                                 void *stream) {
    auto bad = [](const char *what) {
        char buf[256];
        snprintf(buf, sizeof buf, "strata_moe_route_logits: %s", what);
        set_error_message(buf);
        return STRATA_ERR_INVALID_ARG;
    };
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E)
        return bad("need T >= 0, 1 <= E <= 1024, 1 <= k <= min(E, 32)");
    if (logits_type != STRATA_BF16 && logits_type != STRATA_F32)
        return bad("logits_type must be STRATA_BF16 or STRATA_F32");
    if (ld < E) return bad("ld must be at least E");
    SelectPlan plan;
    const strata_status st = make_select_plan(rule, E, k, "strata_moe_route_logits", &plan);
    if (st != STRATA_OK) return st;
    if (T == 0) return STRATA_OK;
    if (!logits_dev || !idx_dev || !w_dev) return bad("NULL device pointer");
    const bool bf16 = logits_type == STRATA_BF16;
    if (((uintptr_t)logits_dev % (bf16 ? 2 : 4)) || ((uintptr_t)select_bias_dev % 4) ||
        ((uintptr_t)idx_dev % 4) || ((uintptr_t)w_dev % 4))
        return bad("misaligned device pointer");
    if (ld > (INT64_MAX / 4) / T) return bad("T * ld is too large");
    const PointerDevice on(logits_dev);
    if (!on.ok) return bad("logits_dev is not device memory");
    plan.bias = select_bias_dev;
    const cudaError_t e = launch_route_logits(plan, logits_dev, bf16, ld, T, idx_dev, w_dev,
                                              (cudaStream_t)stream);
    if (e != cudaSuccess) {
        char buf[256];
        snprintf(buf, sizeof buf, "strata_moe_route_logits: %s", cudaGetErrorString(e));
        set_error_message(buf);
        return STRATA_ERR_CUDA;
    }
    return STRATA_OK;
}
