// Routing rules for many tokens: 8 or 16 lanes a token (select.cuh).
#include "common.cuh"
#include "internal.h"
#include "select.cuh"

namespace strata {

// Lanes of a token.  Fewer lanes share the reductions, ranks and weights among
// more tokens of a warp (791 / 479 / 344 instructions a token of 256 experts with
// 32 / 16 / 8 lanes), but make fewer warps and need more registers: 16 pay from
// 8192 tokens on (4096 of 256 experts: 4.6 us against 3.5 with 32; 8192: 4.8
// against 5.5), 8 from 16384 on (6.9 against 7.3 with 16), and a bias next to
// more than 16 experts a lane spills (16384 tokens of 512 with a bias: 20.5 us
// with 16 lanes, 15.9 with 32).  Two values a lane have to make k of them.
int route_batch_lanes(const SelectPlan &p, int T) {
    const int most = p.bias ? 16 : 32;
    if (p.k > 16 || T < 8192) return 32;
    if (T >= 16384 && lane_elements(p, 8) <= most) return 8;
    return lane_elements(p, 16) <= most ? 16 : 32;
}

cudaError_t launch_route_batch(const SelectPlan &p, const void *logits, bool bf16, long long ld, int T, int32_t *idx,
                               float *w, bool vec, cudaStream_t s) {
    const int lanes = route_batch_lanes(p, T), n = lane_elements(p, lanes);
    if (lanes == 8) {
        if (n <= 8) return run_route<8, 8>(p, logits, bf16, ld, T, idx, w, vec, s);
        if (n <= 16) return run_route<8, 16>(p, logits, bf16, ld, T, idx, w, vec, s);
        return run_route<8, 32, false>(p, logits, bf16, ld, T, idx, w, vec, s);
    }
    if (n <= 8) return run_route<16, 8>(p, logits, bf16, ld, T, idx, w, vec, s);
    if (n <= 16) return run_route<16, 16>(p, logits, bf16, ld, T, idx, w, vec, s);
    return run_route<16, 32, false>(p, logits, bf16, ld, T, idx, w, vec, s);
}

}  // namespace strata
