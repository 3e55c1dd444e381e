// Exact router logits of large batches (layers with a routing rule): the
// fixed-order fp32 dot products of route.cu, bit for bit, from tiles in shared
// memory.
//
//   logit[t][e]: 32 lane partials p_l over i = l, l + 32, ... (fma, ascending i),
//   then p_l += p_{l + s} for s = 16, 8, 4, 2, 1, then + b[e].
//
// T E H multiply-adds on the CUDA cores bound it (10.7 G at T = 8192, E = 512, H =
// 2560: 0.31 ms at 128 a cycle and SM).  A warp holds 8 tokens x 8 experts of
// partials in registers, a block of 16 warps 32 x 32, so a step of 128 columns
// reads 24 KB from L2 for 131 K multiply-adds; steps arrive two at a time, three
// stages ahead (cp.async).  606 us there (912 with route.cu's router, whose rows
// come from L2 again for every 32 experts), the multiply-add pipe throttling:
// 5277 instructions a warp, 2560 of them of two multiply-adds, 710 us and 8417
// with single ones.
#include "common.cuh"
#include "internal.h"

namespace strata {

constexpr int kRtTok = 32, kRtExp = 32, kRtSteps = 2, kRtStages = 4, kRtThreads = 512;
constexpr int kRtX = kRtTok * kRtSteps * 32;  // uint2 of a stage
constexpr int kRtW = kRtExp * kRtSteps * 32;  // float4 of a stage
constexpr int kRtStageBytes = kRtX * 8 + kRtW * 16;

// x [T][H] in the weights' order: xi[t][H / 128][32][4], lane l's four values of a
// step at 128 s + 32 j + l.
__global__ __launch_bounds__(256) void interleave_rows_kernel(const unsigned short *__restrict__ x, long long n,
                                                              uint2 *__restrict__ xi) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // (t, s, lane): 128 columns a warp
    if (i >= n) return;
    const unsigned short *p = x + (i >> 5) * 128 + (i & 31);
    const uint32_t a = p[0], b = p[32], c = p[64], d = p[96];
    xi[i] = make_uint2(a | (b << 16), c | (d << 16));
}

STRATA_DEV void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Two floats (bits) as one operand, and two fused multiply-adds, each rounded as
// fmaf rounds.
STRATA_DEV unsigned long long pack2(uint32_t lo, uint32_t hi) {
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
STRATA_DEV unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__global__ __launch_bounds__(kRtThreads, 1) void router_tile_kernel(const uint2 *__restrict__ xi, int T, int ns4,
                                                                    const float4 *__restrict__ Wp,
                                                                    const float *__restrict__ bias, int E,
                                                                    float *__restrict__ logits) {
    extern __shared__ __align__(16) uint8_t rt_sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t0 = blockIdx.y * kRtTok, e0 = blockIdx.x * kRtExp;
    const int wt = (warp & 3) * 8, we = (warp >> 2) * 8;  // the warp's tokens and experts of the tile
    const int stages = (ns4 + kRtSteps - 1) / kRtSteps;
    // What a thread copies of a stage: byte offsets at step 0 (rows past the end
    // repeat the last one; their results are not stored) and places in the stage.
    constexpr int kXc = kRtTok * kRtSteps * 16 / kRtThreads, kWc = kRtExp * kRtSteps * 32 / kRtThreads;
    uint32_t xo[kXc], wo[kWc];
    const int xs = (tid >> 4) % kRtSteps, ws = (tid >> 5) % kRtSteps;  // the step of the stage
#pragma unroll
    for (int k = 0; k < kXc; k++) {
        const int row = min(t0 + (tid + k * kRtThreads) / (16 * kRtSteps), T - 1);
        xo[k] = ((uint32_t)row * ns4 + xs) * 256 + (tid & 15) * 16;
    }
#pragma unroll
    for (int k = 0; k < kWc; k++) {
        const int row = min(e0 + (tid + k * kRtThreads) / (32 * kRtSteps), E - 1);
        wo[k] = ((uint32_t)row * ns4 + ws) * 512 + lane * 16;
    }
    const uint32_t sm = smem_u32(rt_sm) + tid * 16;
    auto load = [&](int st) {
        if (st < stages) {
            const uint32_t dst = sm + (st % kRtStages) * kRtStageBytes;
            const char *xb = reinterpret_cast<const char *>(xi) + (size_t)st * kRtSteps * 256;
            const char *wb = reinterpret_cast<const char *>(Wp) + (size_t)st * kRtSteps * 512;
            if (st * kRtSteps + xs < ns4)
#pragma unroll
                for (int k = 0; k < kXc; k++) cp_async16(dst + k * kRtThreads * 16, xb + xo[k]);
            if (st * kRtSteps + ws < ns4)
#pragma unroll
                for (int k = 0; k < kWc; k++) cp_async16(dst + kRtX * 8 + k * kRtThreads * 16, wb + wo[k]);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int st = 0; st < kRtStages - 1; st++) load(st);
    // partials of token pairs (2 a, 2 a + 1), so that one instruction adds to two
    unsigned long long acc[4][8];
#pragma unroll
    for (int a = 0; a < 4; a++)
#pragma unroll
        for (int b = 0; b < 8; b++) acc[a][b] = 0ull;
    for (int st = 0; st < stages; st++) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRtStages - 2) : "memory");
        __syncthreads();  // the stage is there for every warp, and the one before it is free
        load(st + kRtStages - 1);
        const uint8_t *base = rt_sm + (st % kRtStages) * kRtStageBytes;
        const uint2 *sx = reinterpret_cast<const uint2 *>(base) + wt * kRtSteps * 32 + lane;
        const float4 *sw = reinterpret_cast<const float4 *>(base + kRtX * 8) + we * kRtSteps * 32 + lane;
        const int cols = min(kRtSteps, ns4 - st * kRtSteps);
        for (int s = 0; s < cols; s++) {
            uint2 x[8];
#pragma unroll
            for (int a = 0; a < 8; a++) x[a] = sx[(a * kRtSteps + s) * 32];
            unsigned long long xp[4][4];  // column j of a token pair
#pragma unroll
            for (int a = 0; a < 4; a++) {
                const uint2 u = x[2 * a], v = x[2 * a + 1];
                xp[a][0] = pack2(u.x << 16, v.x << 16);
                xp[a][1] = pack2(u.x & 0xffff0000u, v.x & 0xffff0000u);
                xp[a][2] = pack2(u.y << 16, v.y << 16);
                xp[a][3] = pack2(u.y & 0xffff0000u, v.y & 0xffff0000u);
            }
#pragma unroll
            for (int b = 0; b < 8; b++) {
                const float4 w = sw[(b * kRtSteps + s) * 32];
                const float wj[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint32_t u = __float_as_uint(wj[j]);
                    const unsigned long long ww = pack2(u, u);
#pragma unroll
                    for (int a = 0; a < 4; a++) acc[a][b] = fma2(xp[a][j], ww, acc[a][b]);
                }
            }
        }
    }
    // the halving tree, two outputs at a time: the lower half of the lanes goes on
    // with one of them, the upper half with the other, so 64 sums take 62
    // exchanges and lane l ends with outputs 2 l and 2 l + 1
    float v[64];
#pragma unroll
    for (int o = 0; o < 64; o++)
        v[o] = __uint_as_float((uint32_t)(acc[o >> 4][o & 7] >> ((o >> 3) & 1 ? 32 : 0)));
#pragma unroll
    for (int s = 16, n = 32; s >= 1; s >>= 1, n >>= 1) {
        const bool upper = lane & s;
#pragma unroll
        for (int o = 0; o < n; o++) {
            const float keep = upper ? v[o + n] : v[o], give = upper ? v[o] : v[o + n];
            v[o] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, s));
        }
    }
    const int t = t0 + wt + lane / 4;
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const int e = e0 + we + (2 * lane + q) % 8;
        if (t < T && e < E) logits[(long long)t * E + e] = bias ? __fadd_rn(v[q], bias[e]) : v[q];
    }
}

void launch_router_tile(const void *x, int T, int H, const float *Wp, const float *bias, int E, void *xi,
                        float *logits, cudaStream_t s) {
    const long long n = (long long)T * (H / 128) * 32;
    interleave_rows_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(reinterpret_cast<const unsigned short *>(x), n,
                                                                      reinterpret_cast<uint2 *>(xi));
    const dim3 grid((E + kRtExp - 1) / kRtExp, (T + kRtTok - 1) / kRtTok);
    router_tile_kernel<<<grid, kRtThreads, kRtStages * kRtStageBytes, s>>>(
        reinterpret_cast<const uint2 *>(xi), T, H / 128, reinterpret_cast<const float4 *>(Wp), bias, E, logits);
}

cudaError_t route_tile_init_attributes(int max_smem) { return allow_max_dyn_smem(router_tile_kernel, max_smem); }

}  // namespace strata
