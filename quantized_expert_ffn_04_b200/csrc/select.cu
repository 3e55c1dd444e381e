// Routing rules: picks and weights from logits (strata_moe_route_logits), and
// the same kernel for a layer whose rule is set (strata_moe_set_routing).
//
// One warp per token here, several tokens a warp in select_batch.cu (select.cuh).
// The work is one read of the logits and a few hundred instructions a token.  In
// large batches the instructions bound it: 65536 tokens of 256 experts (8 groups,
// sigmoid scores with a bias) take 39 us, 481 instructions a token at 74 % of the
// issue slots, where the read alone would take 11; without groups and bias 20.6 us.
// With a token a warp it is the loads' latency first: 8192 tokens of 512 experts
// (sigmoid, bias) take 8.7 us at 57 % of the issue slots (the read: 2.7).
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "select.cuh"

namespace strata {

cudaError_t launch_route_logits(const SelectPlan &p, const void *logits, bool bf16, long long ld,
                                int T, int32_t *idx, float *w, cudaStream_t s) {
    // four logits a load where every group of every row (and the bias) starts at
    // a multiple of it
    const bool vec = p.gs % 4 == 0 && ld % 4 == 0 && ((uintptr_t)logits % (bf16 ? 8 : 16)) == 0 &&
                     ((uintptr_t)p.bias % 16) == 0;
    if (route_batch_lanes(p, T) < 32) return launch_route_batch(p, logits, bf16, ld, T, idx, w, vec, s);
    const int n = lane_elements(p, 32);
    if (n <= 4) return run_route<32, 4>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (n <= 8) return run_route<32, 8>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (n <= 16) return run_route<32, 16>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (n <= 32) return run_route<32, 32>(p, logits, bf16, ld, T, idx, w, vec, s);
    return run_route<32, 64>(p, logits, bf16, ld, T, idx, w, vec, s);  // 1024 / 17 = 60 experts a lane
}

strata_status make_select_plan(const strata_moe_routing *rule, int E, int k, const char *who,
                               SelectPlan *plan) {
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
    if (what) return refuse(who, what);
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
    while ((1 << p.log2_groups) < p.n_groups) p.log2_groups++;
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
    static const char *const who = "strata_moe_route_logits";
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E)
        return refuse(who, "need T >= 0, 1 <= E <= 1024, 1 <= k <= min(E, 32)");
    if (logits_type != STRATA_BF16 && logits_type != STRATA_F32)
        return refuse(who, "logits_type must be STRATA_BF16 or STRATA_F32");
    if (ld < E) return refuse(who, "ld must be at least E");
    SelectPlan plan;
    const strata_status st = make_select_plan(rule, E, k, who, &plan);
    if (st != STRATA_OK) return st;
    if (T == 0) return STRATA_OK;
    if (!logits_dev || !idx_dev || !w_dev) return refuse(who, "NULL device pointer");
    const bool bf16 = logits_type == STRATA_BF16;
    if (((uintptr_t)logits_dev % (bf16 ? 2 : 4)) || ((uintptr_t)select_bias_dev % 4) ||
        ((uintptr_t)idx_dev % 4) || ((uintptr_t)w_dev % 4))
        return refuse(who, "misaligned device pointer");
    if (ld > (INT64_MAX / 4) / T) return refuse(who, "T * ld is too large");
    const int size = bf16 ? 2 : 4;
    const Span in(logits_dev, T, ld * size, (long long)E * size), sb(select_bias_dev, 1, 0, 4ll * E);
    const Span is(idx_dev, 1, 0, 4ll * T * k), ws(w_dev, 1, 0, 4ll * T * k);
    if (is.meets(in) || is.meets(sb) || ws.meets(in) || ws.meets(sb) || is.meets(ws))
        return refuse(who, "an output overlaps another buffer");
    const PointerDevice on(logits_dev);
    if (!on.ok) return refuse(who, "logits_dev is not device memory");
    plan.bias = select_bias_dev;
    return launched(who, launch_route_logits(plan, logits_dev, bf16, ld, T, idx_dev, w_dev, (cudaStream_t)stream));
}
