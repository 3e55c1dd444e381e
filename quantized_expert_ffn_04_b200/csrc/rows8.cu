// 8-bit rows: the block's pre-norm that writes them (residual addition,
// weighted RMSNorm, quantisation) and the row gather that reads them back.
//
//   h = bf16(x + delta);  y = h r w,  r = 1 / sqrt(mean(h^2) + eps);
//   a group's scale s = max|y| / M (M = 448 for e4m3, 127 for int8);
//   code = round(y M / max|y|);  read back: bf16(code s).
//
// Both kernels are one pass over HBM.
#include <float.h>
#include <math.h>
#include <stdio.h>

#include "common.cuh"
#include "internal.h"

namespace strata {

constexpr float kE4m3Max = 448.0f;
constexpr float kInt8Max = 127.0f;
// A group whose largest magnitude is below this stores zeros: its scale and
// the reciprocal of it would leave fp32's normal range (448 / 2^-116 < 2^125).
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
    int T, H, group, weight_f32;
};

// Reduce over the block's kThreads threads; every thread gets the result.
template <int kThreads, typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V *scratch, F op) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (kThreads == 32) return v;
    const int warp = threadIdx.x >> 5;
    __syncthreads();  // the scratch's previous use
    if ((threadIdx.x & 31) == 0) scratch[warp] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; i++) v = op(v, scratch[i]);
    return v;
}

// One block per row; thread i holds the 16-byte vectors i, i + kThreads, ...
template <int kThreads, int NV, int kQ8, bool kF32Weight>
__global__ __launch_bounds__(kThreads) void add_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float fs[kThreads / 32];
    __shared__ uint32_t us[kThreads / 32];
    __shared__ double ds[kThreads / 32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int nv = a.H >> 3, tid = threadIdx.x;
    const long long row = (long long)blockIdx.x * nv;
    uint4 hv[NV], dv[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = i * kThreads + tid;
        hv[i] = c < nv ? a.x[row + c] : make_uint4(0, 0, 0, 0);
        dv[i] = a.delta && c < nv ? a.delta[row + c] : make_uint4(0, 0, 0, 0);
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = i * kThreads + tid;
        float f[8], d[8];
        unpack8(hv[i], f);
        if (a.delta) {
            unpack8(dv[i], d);
#pragma unroll
            for (int q = 0; q < 8; q++) f[q] = __fadd_rn(f[q], d[q]);
            hv[i] = pack8(f);
            unpack8(hv[i], f);
        }
        if (a.h_out && c < nv) a.h_out[row + c] = hv[i];
#pragma unroll
        for (int q = 0; q < 8; q++) ss = fmaf(f[q], f[q], ss);
    }
    auto add = [](float p, float q) { return p + q; };
    auto umax = [](uint32_t p, uint32_t q) { return p > q ? p : q; };
    ss = block_reduce<kThreads>(ss, fs, add);
    // r = 1 / sqrt(mean + eps) as unit * rr: 64 bits where the squares' sum
    // leaves fp32's range (unit a power of two, so that both are normal floats)
    float unit = 1.0f, rr;
    if ((ss < 1e-30f && a.eps < 1e-30f) || !(ss < 1e37f)) {
        double sd = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float f[8];
            unpack8(hv[i], f);
#pragma unroll
            for (int q = 0; q < 8; q++) sd = fma((double)f[q], (double)f[q], sd);
        }
        sd = block_reduce<kThreads>(sd, ds, [](double p, double q) { return p + q; });
        const double r = 1.0 / sqrt(sd / a.H + (double)a.eps);
        const int ex = r > 0.0 && r < INFINITY ? max(-126, min(126, ilogb(r))) : 0;
        unit = __uint_as_float((uint32_t)(127 + ex) << 23);
        rr = (float)(r / (double)unit);
    } else {
        rr = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, a.inv_h, a.eps)));
    }
    uint32_t row_max = 0;
    float inv = 0.0f;
    auto values = [&](int i, float (&y)[8]) {  // y of vector i
        const int c = i * kThreads + tid;
        float w[8];
#pragma unroll
        for (int q = 0; q < 8; q++) w[q] = 1.0f;
        if (a.weight && c < nv) {
            if (kF32Weight) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * c);
                const float4 v = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * c + 1);
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
            } else {
                unpack8(__ldg(reinterpret_cast<const uint4 *>(a.weight) + c), w);
            }
        }
        unpack8(hv[i], y);
#pragma unroll
        for (int q = 0; q < 8; q++) y[q] = (y[q] * unit) * rr * w[q];
    };
    auto emit = [&](int i, const float (&y)[8], float mul) {
        const int c = i * kThreads + tid;
        if (c >= nv) return;
        uint2 o;
        o.x = codes4<kQ8>(y[0] * mul, y[1] * mul, y[2] * mul, y[3] * mul);
        o.y = codes4<kQ8>(y[4] * mul, y[5] * mul, y[6] * mul, y[7] * mul);
        if (mul == 0.0f) o = make_uint2(0, 0);  // also where a value is not finite
        *reinterpret_cast<uint2 *>(a.q + (long long)blockIdx.x * a.q_stride + 8 * c) = o;
    };
    constexpr float kMax = kQ8 == STRATA_Q8_E4M3 ? kE4m3Max : kInt8Max;
    // group maximum (float bits; a NaN is above all) -> stored scale and multiplier
    auto scale_of = [&](uint32_t bits, float &mul) {
        const float m = __uint_as_float(bits);
        if (bits >= 0x7f800000u) {
            mul = 0.0f;
            return __uint_as_float(0x7fc00000u);
        }
        mul = m < kTinyGroup ? 0.0f : __fdiv_rn(kMax, m);
        return m < kTinyGroup ? 0.0f : __fdiv_rn(m, kMax);
    };
    float *srow = a.q ? a.scale + (long long)blockIdx.x * a.scale_stride : nullptr;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = i * kThreads + tid;
        float y[8];
        values(i, y);
        if (a.xn && c < nv) a.xn[row + c] = pack8(y);
        if (!a.q) continue;
        uint32_t am = 0;
#pragma unroll
        for (int q = 0; q < 8; q++) am = umax(am, __float_as_uint(y[q]) & 0x7fffffffu);
        if (a.group) {
            // group / 8 neighbouring threads hold a group
            for (int o = a.group >> 4; o >= 1; o >>= 1) am = umax(am, __shfl_xor_sync(0xffffffffu, am, o));
            float mul;
            const float sc = scale_of(am, mul);
            if (c < nv && 8 * c % a.group == 0) srow[8 * c / a.group] = sc;
            emit(i, y, mul);
        } else {
            row_max = umax(row_max, c < nv ? am : 0u);
        }
    }
    if (a.q && !a.group) {
        row_max = block_reduce<kThreads>(row_max, us, umax);
        const float sc = scale_of(row_max, inv);
        if (tid == 0) srow[0] = sc;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float y[8];
            values(i, y);
            emit(i, y, inv);
        }
    }
}

template <int NV, int kQ8, bool kF32Weight>
static cudaError_t run_norm(const NormArgs &a, cudaStream_t s) {
    return launch_pdl(add_rmsnorm_kernel<128, NV, kQ8, kF32Weight>, dim3(a.T), dim3(128), 0, s, a);
}
template <int kQ8, bool kF32Weight>
static cudaError_t run_norm_nv(const NormArgs &a, cudaStream_t s) {
    const int nv = (a.H / 8 + 127) / 128;
    if (nv <= 1) return run_norm<1, kQ8, kF32Weight>(a, s);
    if (nv <= 2) return run_norm<2, kQ8, kF32Weight>(a, s);
    if (nv <= 3) return run_norm<3, kQ8, kF32Weight>(a, s);
    if (nv <= 4) return run_norm<4, kQ8, kF32Weight>(a, s);
    if (nv <= 6) return run_norm<6, kQ8, kF32Weight>(a, s);
    if (nv <= 8) return run_norm<8, kQ8, kF32Weight>(a, s);
    return run_norm<16, kQ8, kF32Weight>(a, s);
}

static cudaError_t launch_add_rmsnorm(const NormArgs &a, int q8, cudaStream_t s) {
    if (q8 == STRATA_Q8_INT8)
        return a.weight_f32 ? run_norm_nv<STRATA_Q8_INT8, true>(a, s) : run_norm_nv<STRATA_Q8_INT8, false>(a, s);
    return a.weight_f32 ? run_norm_nv<STRATA_Q8_E4M3, true>(a, s) : run_norm_nv<STRATA_Q8_E4M3, false>(a, s);
}

// ------------------------------------------------------------------ read back
struct DequantArgs {
    const uint8_t *q;
    const float *scale;
    const int32_t *rows;
    uint4 *out;
    long long q_stride, scale_stride;
    int group, n, n_src, H;
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

// One warp per row; a lane turns 16 codes into 32 bytes.
template <int kQ8>
__global__ __launch_bounds__(128) void dequant_rows_kernel(const __grid_constant__ DequantArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= a.n) return;
    const int r = a.rows ? a.rows[i] : i;
    if ((unsigned)r >= (unsigned)a.n_src) return;
    const uint8_t *q = a.q + (long long)r * a.q_stride;
    const float *sc = a.scale + (long long)r * a.scale_stride;
    uint4 *o = a.out + (long long)i * (a.H >> 3);
    for (int c = lane; c < (a.H >> 4); c += 32) {
        const uint4 u = *reinterpret_cast<const uint4 *>(q + 16 * c);
        const float s = sc[a.group ? 16 * c / a.group : 0];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float f[16];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            float g[4];
            values4<kQ8>(w[k], g);
#pragma unroll
            for (int j = 0; j < 4; j++) f[4 * k + j] = g[j] * s;
        }
        float lo[8], hi[8];
#pragma unroll
        for (int k = 0; k < 8; k++) lo[k] = f[k], hi[k] = f[8 + k];
        o[2 * c] = pack8(lo);
        o[2 * c + 1] = pack8(hi);
    }
}

static cudaError_t launch_dequant_rows(const DequantArgs &a, int q8, cudaStream_t s) {
    const dim3 grid((unsigned)((a.n + 3) / 4));
    return launch_pdl(q8 == STRATA_Q8_INT8 ? dequant_rows_kernel<STRATA_Q8_INT8> : dequant_rows_kernel<STRATA_Q8_E4M3>,
                      grid, dim3(128), 0, s, a);
}

// A call's refusal: message and status.
static strata_status refuse(const char *who, const char *what) {
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", who, what);
    set_error_message(buf);
    return STRATA_ERR_INVALID_ARG;
}
static strata_status launched(const char *who, cudaError_t e) {
    if (e == cudaSuccess) return STRATA_OK;
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", who, cudaGetErrorString(e));
    set_error_message(buf);
    return STRATA_ERR_CUDA;
}

// A caller's buffer of `rows` rows of `bytes` bytes, `stride` bytes apart.
struct Span {
    uintptr_t begin = 0, end = 0;
    Span(const void *p, long long rows, long long stride, long long bytes) {
        if (!p || rows <= 0) return;
        begin = (uintptr_t)p;
        end = begin + (uintptr_t)((rows - 1) * stride + bytes);
    }
    bool meets(const Span &o) const { return begin < o.end && o.begin < end; }
};

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
    a.group = q_dev ? group : 0;
    a.weight_f32 = weight_type == STRATA_F32;
    return launched(who, launch_add_rmsnorm(a, q_dev ? q8 : STRATA_Q8_E4M3, (cudaStream_t)stream));
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
    a.group = group;
    a.n = n;
    a.n_src = n_src;
    a.H = H;
    return launched(who, launch_dequant_rows(a, q8, (cudaStream_t)stream));
}

}  // extern "C"
