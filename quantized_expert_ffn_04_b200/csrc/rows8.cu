// 8-bit rows: the block's pre-norm that writes them (residual addition,
// weighted RMSNorm, quantisation) and the row gather that reads them back.
//
//   h = bf16(x + delta);  y = h r w,  r = 1 / sqrt(mean(h^2) + eps);
//   a group's scale s = max|y| / M (M = 448 for e4m3, 127 for int8);
//   code = round(y M / max|y|);  read back: bf16(code s).
//
// Both kernels are one pass over HBM, which bounds them at prompt sizes: 8192 rows
// of 2560 (x, delta in; h, xn, e4m3 codes out: 189 MB) 33 us, with inputs that left
// L2, where a copy's rate gives 28.9; 81920 rows read (441 MB, 420 of them written)
// 74 us where it gives 67 (64 back to back, a fill of the output alone 60).  One to
// 64 rows take 2.2 to 2.5 us, a launch.
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace strata {

constexpr float kE4m3Max = 448.0f;
constexpr float kInt8Max = 127.0f;
constexpr int kNormThreads = 1024;
// A group whose largest magnitude is below this stores zeros: its scale would
// leave fp32's normal range (2^-116 / 448 > 2^-125).
constexpr float kTinyGroup = 1.2037062e-35f;  // 2^-116

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
// bf16(f32(x) + f32(d)) of eight pairs.  One rounded bf16 addition gives the same:
// fp32 rounds the sum only where d is below 2^-16 of x (or x of d), and there
// both forms return the larger of the two.
__device__ __forceinline__ uint4 add8(const uint4 &x, const uint4 &d) {
    auto add = [](uint32_t p, uint32_t q) {
        const __nv_bfloat162 v = __hadd2_rn(*reinterpret_cast<__nv_bfloat162 *>(&p), *reinterpret_cast<__nv_bfloat162 *>(&q));
        return *reinterpret_cast<const uint32_t *>(&v);
    };
    return make_uint4(add(x.x, d.x), add(x.y, d.y), add(x.z, d.z), add(x.w, d.w));
}
// Four values to four codes; the first in the lowest byte.
template <int kQ8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    if (kQ8 == STRATA_Q8_E4M3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    const int i = __float2int_rn(a), j = __float2int_rn(b), k = __float2int_rn(c), l = __float2int_rn(d);
    const uint32_t lo = __byte_perm((uint32_t)i, (uint32_t)j, 0x0040);  // i0 j0 . .
    const uint32_t hi = __byte_perm((uint32_t)k, (uint32_t)l, 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// ------------------------------------------------------------------ add + RMSNorm
struct NormArgs {
    const uint4 *x, *delta;
    const void *weight;
    uint4 *h_out, *xn;
    uint8_t *q;
    float *scale;
    long long q_stride, scale_stride;
    float eps, inv_h;
    int T, H, weight_f32;
};

// Largest of two magnitudes; a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Sum over the row's 32-vector blocks: v[i] is this thread's part of block
// i * warps + warp.  A tree inside each block, then one over the blocks, so the
// sum does not depend on how many vectors a thread holds.
template <int NV, typename V>
__device__ __forceinline__ V row_sum(V (&v)[NV], V *scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < NV; i++) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lane == 0) scratch[i * warps + warp] = v[i];
    }
    __syncthreads();
    const int blocks = NV * warps;
    V sum = lane < blocks ? scratch[lane] : (V)0;
    if (NV > 1) sum += lane + 32 < blocks ? scratch[lane + 32] : (V)0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
__device__ __forceinline__ float row_max(float v, float *scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0) scratch[warp] = v;
    __syncthreads();
    v = scratch[lane < warps ? lane : 0];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// One row a block; thread i holds the 16-byte vectors i and (NV == 2)
// i + blockDim.x, so that the row stays in registers between its one read and its
// one write (a warp a row needs 10 vectors a thread: 46 to 58 us for 8192 rows of
// 2560).  261 instructions a vector; the issue slots are 72 % taken.  kGroup: columns
// a scale covers, 0 for the whole row, -1 for no 8-bit output.
template <int NV, int kQ8, int kGroup, bool kF32Weight>
__global__ __launch_bounds__(kNormThreads) void add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float fs[64], ms[32];
    __shared__ double ds[64];
    grid_launch_dependents();
    grid_dependency_wait();
    const int nv = a.H >> 3, tid = threadIdx.x, threads = blockDim.x;
    const long long t = blockIdx.x, row = t * nv;
    uint4 hv[NV], dv[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = i * threads + tid;
        hv[i] = c < nv ? a.x[row + c] : make_uint4(0, 0, 0, 0);
        if (a.delta) dv[i] = c < nv ? a.delta[row + c] : make_uint4(0, 0, 0, 0);
    }
    float h[NV][8], part[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = i * threads + tid;
        if (a.delta) hv[i] = add8(hv[i], dv[i]);
        if (a.h_out && c < nv) a.h_out[row + c] = hv[i];
        unpack8(hv[i], h[i]);
        part[i] = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; q++) part[i] = fmaf(h[i][q], h[i][q], part[i]);
    }
    const float ss = row_sum<NV>(part, fs);
    // r = 1 / sqrt(mean + eps), in 64 bits where the squares' sum comes near the
    // ends of fp32's range.  A factor above 2 is split: its power of two goes into
    // h, exactly (|h| r <= sqrt(H)), and r stays in [1, 2).  So t = h w below is
    // within a factor of 2 of y = t r (or above it), and leaves fp32's normal range
    // only where y does.
    float r = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, a.inv_h, a.eps)));
    float late = 1.0f;  // below 1: the power of two of a small r, see times_late
    int ex = 0;
    if ((ss < 0x1p-60f && a.eps < 0x1p-60f) || !(ss < 0x1p60f)) {
        double dp[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            dp[i] = 0.0;
#pragma unroll
            for (int q = 0; q < 8; q++) dp[i] = fma((double)h[i][q], (double)h[i][q], dp[i]);
        }
        const double rd = 1.0 / sqrt(row_sum<NV>(dp, ds) / a.H + (double)a.eps);
        ex = rd > 0.0 && rd < INFINITY ? max(-126, ilogb(rd)) : 0;  // at most 140
        r = (float)scalbn(rd, -ex);
        if (ex < 0) late = pow2(ex);
    } else if (r >= 2.0f) {
        ex = (int)(__float_as_uint(r) >> 23) - 127;
        r *= pow2(-ex);
    }
    if (ex > 0) {
        const float up = pow2(min(ex, 126)), rest = pow2(max(ex, 126) - 126);
#pragma unroll
        for (int i = 0; i < NV; i++)
#pragma unroll
            for (int q = 0; q < 8; q++) h[i][q] = h[i][q] * up * rest;
    }
    // h w 2^ex for ex < 0: the power first where h is large (h w might overflow), last
    // where it is not (h 2^ex might underflow)
    auto times_late = [&](float v, float w) {
        const bool first = fabsf(v) >= 1.0f;
        return v * (first ? late : 1.0f) * w * (first ? 1.0f : late);
    };
    constexpr float kMax = kQ8 == STRATA_Q8_E4M3 ? kE4m3Max : kInt8Max;
    // y = t r with t = h w (exact for bf16 weights).  A code is the rounded
    // quotient kMax t / max|t|: (c t) / m with m = max|t| scaled into [1, 2) and c
    // = kMax times the same power of two, both exact where t is (y >= 2^-116 and r <=
    // 2 leave max|t| >= 2^-117, so c <= 448 2^117).  The quotient is
    // corrected once by its remainder (Markstein's method), which makes it exact
    // where it is representable: a value exactly between two codes goes to the
    // even one, as it does in 64 bits.
    struct Group {
        float c, m, inv;
    };
    auto group_of = [&](float mt, float &scale) {
        const float y = mt * r;
        Group g{0.0f, 1.0f, 1.0f};
        scale = y * (1.0f / kMax);
        if (y >= kTinyGroup && y < INFINITY) {
            const uint32_t bits = __float_as_uint(mt);
            g.m = __uint_as_float((bits & 0x007fffffu) | 0x3f800000u);
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.m));
            g.c = __uint_as_float(__float_as_uint(kMax) + ((127u - (bits >> 23)) << 23));
        } else {
            scale = y < INFINITY ? 0.0f : __uint_as_float(0x7fc00000u);
        }
        return g;
    };
    auto emit = [&](int i, const Group &g) {
        const int c = i * threads + tid;
        float k[8];
#pragma unroll
        for (int q = 0; q < 8; q++) {
            const float n = h[i][q] * g.c, q0 = n * g.inv;
            k[q] = fmaf(fmaf(-g.m, q0, n), g.inv, q0);
        }
        uint2 o = make_uint2(codes4<kQ8>(k[0], k[1], k[2], k[3]), codes4<kQ8>(k[4], k[5], k[6], k[7]));
        if (g.c == 0.0f) o = make_uint2(0, 0);  // also where a value is not finite
        if (c < nv) *reinterpret_cast<uint2 *>(a.q + t * a.q_stride + 8 * c) = o;
    };
    float largest = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = i * threads + tid;
        if (a.weight && c < nv) {
            float w[8];
            if (kF32Weight) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * c);
                const float4 v = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * c + 1);
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
            } else {
                unpack8(__ldg(reinterpret_cast<const uint4 *>(a.weight) + c), w);
            }
            if (late == 1.0f) {
#pragma unroll
                for (int q = 0; q < 8; q++) h[i][q] *= w[q];
            } else {
#pragma unroll
                for (int q = 0; q < 8; q++) h[i][q] = times_late(h[i][q], w[q]);
            }
        } else if (late < 1.0f) {
#pragma unroll
            for (int q = 0; q < 8; q++) h[i][q] *= late;
        }
        if (a.xn && c < nv) {
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; q++) o[q] = h[i][q] * r;
            a.xn[row + c] = pack8(o);
        }
        if (kGroup < 0) continue;
        float m = fabsf(h[i][0]);
#pragma unroll
        for (int q = 1; q < 8; q++) m = max_nan(m, fabsf(h[i][q]));
        if (kGroup > 0) {
            // kGroup / 8 neighbouring threads hold a group
#pragma unroll
            for (int o = kGroup / 16; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            float scale;
            const Group g = group_of(m, scale);
            constexpr int kVecs = kGroup > 0 ? kGroup / 8 : 1;
            if (c < nv && c % kVecs == 0) a.scale[t * a.scale_stride + c / kVecs] = scale;
            emit(i, g);
        } else {
            largest = max_nan(largest, m);  // a vector past the row holds zeros
        }
    }
    if (kGroup == 0) {
        float scale;
        const Group g = group_of(row_max(largest, ms), scale);
        if (tid == 0) a.scale[t * a.scale_stride] = scale;
#pragma unroll
        for (int i = 0; i < NV; i++) emit(i, g);
    }
}

template <int kQ8, int kGroup, bool kF32Weight>
static cudaError_t run_norm(const NormArgs &a, cudaStream_t s) {
    const int nv = a.H / 8;
    // One vector a thread while a row finds an SM of its own (148 of them): the
    // row's latency is all that counts (64 rows of 2560: 2.3 us, 2.8 with two).
    // Two above, so that more rows are in flight and the block's reduction is
    // shared by more work (4001 rows: 16.2 us, 17.2 with one; 333 of 6144: 4.4,
    // 4.8).
    if (a.T <= 148 && nv <= kNormThreads)
        return launch_pdl(add_rmsnorm_kernel<1, kQ8, kGroup, kF32Weight>, dim3(a.T), dim3((nv + 31) / 32 * 32), 0, s, a);
    return launch_pdl(add_rmsnorm_kernel<2, kQ8, kGroup, kF32Weight>, dim3(a.T), dim3((nv / 2 + 31) / 32 * 32), 0, s, a);
}
template <int kQ8>
static cudaError_t run_norm_group(const NormArgs &a, int group, cudaStream_t s) {
    switch (group) {
    case 0: return a.weight_f32 ? run_norm<kQ8, 0, true>(a, s) : run_norm<kQ8, 0, false>(a, s);
    case 32: return a.weight_f32 ? run_norm<kQ8, 32, true>(a, s) : run_norm<kQ8, 32, false>(a, s);
    case 64: return a.weight_f32 ? run_norm<kQ8, 64, true>(a, s) : run_norm<kQ8, 64, false>(a, s);
    default: return a.weight_f32 ? run_norm<kQ8, 128, true>(a, s) : run_norm<kQ8, 128, false>(a, s);
    }
}

static cudaError_t launch_add_rmsnorm(const NormArgs &a, int q8, int group, cudaStream_t s) {
    if (!a.q) return a.weight_f32 ? run_norm<STRATA_Q8_E4M3, -1, true>(a, s) : run_norm<STRATA_Q8_E4M3, -1, false>(a, s);
    return q8 == STRATA_Q8_INT8 ? run_norm_group<STRATA_Q8_INT8>(a, group, s) : run_norm_group<STRATA_Q8_E4M3>(a, group, s);
}

// ------------------------------------------------------------------ read back
struct DequantArgs {
    const uint8_t *q;
    const float *scale;
    const int32_t *rows;
    uint4 *out;
    long long q_stride, scale_stride;
    int log2_group, n, n_src, H;  // log2_group 31: one scale a row
};

// Four codes as floats.
template <int kQ8>
__device__ __forceinline__ void values4(uint32_t u, float (&f)[4]) {
    if (kQ8 == STRATA_Q8_E4M3) {
        uint32_t lo, hi;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(u & 0xffffu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(u >> 16)));
        const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    } else {
        // byte b as 2^23 + (b + 128), less 2^23 + 128: exact
        const uint32_t v = u ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; i++)
            f[i] = __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7440 + i)) - 8388736.0f;
    }
}

// One warp per row, a lane turns 8 codes (one load) into 16 bytes (one store),
// so that both are contiguous over the warp (16 codes a lane leave half sectors in
// every store: 115 us for 81920 rows of 2560 instead of 76), kAhead loads before
// the first store (10: 63.5 us, 5: 64.8).  Streaming stores: the output leaves L2
// first and the source rows, read about ten times each, stay (76 -> 65 us).
constexpr int kDequantWarps = 4, kAhead = 10;
template <int kQ8>
__global__ __launch_bounds__(32 * kDequantWarps) void dequant_rows_kernel(const __grid_constant__ DequantArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * kDequantWarps + (threadIdx.x >> 5);
    if (i >= a.n) return;
    const int r = a.rows ? a.rows[i] : (int)i;
    if ((unsigned)r >= (unsigned)a.n_src) return;
    const int nv = a.H >> 3;
    const uint2 *q = reinterpret_cast<const uint2 *>(a.q + (long long)r * a.q_stride);
    const float *sc = a.scale + (long long)r * a.scale_stride;
    uint4 *o = a.out + i * nv;
    for (int c0 = lane; c0 < nv; c0 += 32 * kAhead) {
        uint2 u[kAhead];
        float s[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int c = c0 + 32 * k;
            u[k] = c < nv ? q[c] : make_uint2(0, 0);
            s[k] = c < nv ? sc[(8 * c) >> a.log2_group] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int c = c0 + 32 * k;
            float lo[4], hi[4];
            values4<kQ8>(u[k].x, lo);
            values4<kQ8>(u[k].y, hi);
            const float f[8] = {lo[0] * s[k], lo[1] * s[k], lo[2] * s[k], lo[3] * s[k],
                                hi[0] * s[k], hi[1] * s[k], hi[2] * s[k], hi[3] * s[k]};
            if (c < nv) __stcs(o + c, pack8(f));
        }
    }
}

static cudaError_t launch_dequant_rows(const DequantArgs &a, int q8, cudaStream_t s) {
    const dim3 grid((unsigned)(((long long)a.n + kDequantWarps - 1) / kDequantWarps));
    return launch_pdl(q8 == STRATA_Q8_INT8 ? dequant_rows_kernel<STRATA_Q8_INT8> : dequant_rows_kernel<STRATA_Q8_E4M3>,
                      grid, dim3(32 * kDequantWarps), 0, s, a);
}

static const char *bad_group(int q8, int group, int H) {
    if (q8 != STRATA_Q8_E4M3 && q8 != STRATA_Q8_INT8) return "q8 must be STRATA_Q8_E4M3 or STRATA_Q8_INT8";
    if (group != 0 && group != 32 && group != 64 && group != 128) return "group must be 0, 32, 64 or 128";
    if (group && H % group) return "group must divide H";
    return nullptr;
}

}  // namespace strata

using namespace strata;

extern "C" {

strata_status strata_moe_add_rmsnorm(const void *x_dev, const void *delta_dev,
                                     const void *weight_dev, int weight_type, float eps, int T,
                                     int H, void *h_out_dev, void *xn_dev, int q8, int group,
                                     void *q_dev, int64_t q_stride, float *scale_dev,
                                     int64_t scale_stride, void *stream) {
    static const char *const who = "strata_moe_add_rmsnorm";
    if (T < 0 || H < 32 || H % 32 || H > 16384) return refuse(who, "need T >= 0 and H a multiple of 32 up to 16384");
    if (weight_type != STRATA_BF16 && weight_type != STRATA_F32)
        return refuse(who, "weight_type must be STRATA_BF16 or STRATA_F32");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return refuse(who, "eps must be finite and >= 0");
    const int n_scales = q_dev && group > 0 ? H / group : 1;
    if (q_dev) {
        if (const char *what = bad_group(q8, group, H)) return refuse(who, what);
        if (q_stride < H || q_stride % 16) return refuse(who, "q_stride must be a multiple of 16 and at least H");
        if (scale_stride < n_scales) return refuse(who, "scale_stride is smaller than a row's scales");
        if (T > 0 && (q_stride > INT64_MAX / 8 / T || scale_stride > INT64_MAX / 8 / T))
            return refuse(who, "a stride is too large");
    }
    if (T == 0) return STRATA_OK;
    if (!x_dev) return refuse(who, "x_dev is NULL");
    if (delta_dev && !h_out_dev) return refuse(who, "h_out_dev is needed with delta_dev");
    if (!h_out_dev && !xn_dev && !q_dev) return refuse(who, "no output buffer");
    if (q_dev && !scale_dev) return refuse(who, "scale_dev is NULL");
    if (!q_dev) scale_dev = nullptr;
    if (((uintptr_t)x_dev | (uintptr_t)delta_dev | (uintptr_t)weight_dev | (uintptr_t)h_out_dev |
         (uintptr_t)xn_dev | (uintptr_t)q_dev | (uintptr_t)scale_dev) & 15)
        return refuse(who, "pointers must be 16-byte aligned");
    const long long rb = (long long)H * 2;
    const Span in[3] = {Span(x_dev, T, rb, rb), Span(delta_dev, T, rb, rb),
                        Span(weight_dev, 1, 0, (long long)H * (weight_type == STRATA_F32 ? 4 : 2))};
    const Span ho(h_out_dev, T, rb, rb), xn(xn_dev, T, rb, rb), qs(q_dev, T, q_stride, H),
        ss(scale_dev, T, 4 * scale_stride, 4 * n_scales);
    for (int i = 0; i < 3; i++)
        if ((ho.meets(in[i]) && !(i == 0 && h_out_dev == x_dev)) || xn.meets(in[i]) || qs.meets(in[i]) || ss.meets(in[i]))
            return refuse(who, "an output overlaps an input");
    // codes and scales may share rows: scales behind the codes of a packed row
    const bool packed = q_dev && q_stride == 4 * scale_stride && (const char *)scale_dev >= (const char *)q_dev + H &&
                        (const char *)(scale_dev + n_scales) <= (const char *)q_dev + q_stride;
    if (ho.meets(xn) || ho.meets(qs) || ho.meets(ss) || xn.meets(qs) || xn.meets(ss) || (qs.meets(ss) && !packed))
        return refuse(who, "two outputs overlap");
    const PointerDevice on(x_dev);
    if (!on.ok) return refuse(who, "x_dev is not device memory");
    NormArgs a{};
    a.x = (const uint4 *)x_dev;
    a.delta = (const uint4 *)delta_dev;
    a.weight = weight_dev;
    a.h_out = (uint4 *)h_out_dev;
    a.xn = (uint4 *)xn_dev;
    a.q = (uint8_t *)q_dev;
    a.scale = scale_dev;
    a.q_stride = q_stride;
    a.scale_stride = scale_stride;
    a.eps = eps;
    a.inv_h = 1.0f / (float)H;
    a.T = T;
    a.H = H;
    a.weight_f32 = weight_type == STRATA_F32;
    return launched(who, launch_add_rmsnorm(a, q8, group, (cudaStream_t)stream));
}

strata_status strata_moe_dequant_rows(const void *q_dev, int q8, int64_t q_stride,
                                      const float *scale_dev, int64_t scale_stride, int group,
                                      const int32_t *rows_dev, int n, int n_src, int H,
                                      void *out_dev, void *stream) {
    static const char *const who = "strata_moe_dequant_rows";
    if (n < 0 || n_src < 0 || H < 32 || H % 32 || H > 65536)
        return refuse(who, "need n >= 0, n_src >= 0 and H a multiple of 32 up to 65536");
    if (const char *what = bad_group(q8, group, H)) return refuse(who, what);
    const int n_scales = group ? H / group : 1;
    if (q_stride < H || q_stride % 16) return refuse(who, "q_stride must be a multiple of 16 and at least H");
    if (scale_stride < n_scales) return refuse(who, "scale_stride is smaller than a row's scales");
    if (n_src > 0 && (q_stride > INT64_MAX / 8 / n_src || scale_stride > INT64_MAX / 8 / n_src))
        return refuse(who, "a stride is too large");
    if (!rows_dev && n > n_src) return refuse(who, "n exceeds n_src without rows_dev");
    if (n == 0 || n_src == 0) return STRATA_OK;
    if (!q_dev || !scale_dev || !out_dev) return refuse(who, "NULL device pointer");
    if ((((uintptr_t)q_dev | (uintptr_t)out_dev) & 15) || (((uintptr_t)scale_dev | (uintptr_t)rows_dev) & 3))
        return refuse(who, "q_dev and out_dev must be 16-byte aligned, scale_dev and rows_dev 4-byte aligned");
    const Span out(out_dev, n, (long long)H * 2, (long long)H * 2);
    if (out.meets(Span(q_dev, n_src, q_stride, H)) || out.meets(Span(scale_dev, n_src, 4 * scale_stride, 4 * n_scales)) ||
        out.meets(Span(rows_dev, n, 4, 4)))
        return refuse(who, "out_dev overlaps an input");
    const PointerDevice on(q_dev);
    if (!on.ok) return refuse(who, "q_dev is not device memory");
    DequantArgs a{};
    a.q = (const uint8_t *)q_dev;
    a.scale = scale_dev;
    a.rows = rows_dev;
    a.out = (uint4 *)out_dev;
    a.q_stride = q_stride;
    a.scale_stride = scale_stride;
    a.log2_group = group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : 31;
    a.n = n;
    a.n_src = n_src;
    a.H = H;
    return launched(who, launch_dequant_rows(a, q8, (cudaStream_t)stream));
}

}  // extern "C"
