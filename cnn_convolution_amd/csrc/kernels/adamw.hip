// One AdamW step over many tensors (im2win_block.h), states in 32 or in 8 bits, and
// the values of 8-bit states. 32 bits are bound by HBM: every element of p, g, m and v is
// read and of p, m and v written once; 8 bits by the VALU and by how launches begin and end.
//
// A launch takes up to kAdamTensors tensors by value, a workgroup one chunk of
// consecutive elements of one of them, a lane 8 (8 bits: 4) consecutive ones: a wave
// holds a block of 256 of an 8-bit state, whose scale is a maximum over its lanes, so the
// states need one pass and no LDS. (With 4 elements a lane 32-bit states take 1152 us for
// 1100 over 200 million; 8-bit ones took 306 us with 8 and 218 with 4, for want of waves.)
// The types of p and g are a workgroup's affair: it branches once to the code for its
// tensor's, so that all loads go out together.
// 200 million elements, fp32 states, bf16 gradients and copies: 1091 us (5.1 TB/s). 40
// million with 8-bit states in one tensor: 157 us (4.0 TB/s), in which the VALU is at work at
// least 85 % of the SIMDs' cycles (472 instructions to a wave's 256 elements, counted as 4
// cycles each; those of fp64 and the square roots take longer). 83 registers let a SIMD have 5
// waves, of which 3.9 are there on average. In 150 tensors 197 us: four launches of 24 to 62
// us in turn, with 60 to 65 % in the larger ones.
//
// 8-bit states: m, v and the scales are formed in fp64, so that the level that an element
// gets is the definition's but for fp64's own roundings. A value in units of its
// block's scale, x = |m| 127^2 / M or v 255^4 / V, lies between c^2 and (c + 1)^2 (fourth
// powers for v), and goes to the upper one if 65536 times its share of the interval
// exceeds its number u. fp32 decides that (c from square roots) unless the two are within
// fp32's error of each other, one element in some ten thousands, for which fp64 does.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../block_launch.hpp"
#include "head_vec.hpp"
#include "philox.hpp"

namespace im2win {
namespace {

constexpr int kThreads = 256;
template <int BITS>
constexpr int kLaneOf = int(adam_chunk(BITS)) / kThreads;    // elements of a lane

template <typename F>
__device__ __forceinline__ void with_type(int t, F f)
{
    if (t == 0)
        f(float{});
    else if (t == 1)
        f(_Float16{});
    else
        f(__bf16{});
}

// 1 - beta^t in fp64
__device__ __forceinline__ double correction(double beta, int64_t t)
{
    return beta > 0.0 ? -expm1(double(t) * log(beta)) : 1.0;
}

// largest of a wave (of |values| as bits: NaN and infinity are above all)
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    auto dpp = [](uint32_t x, auto ctrl) {
        return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    using std::integral_constant;
    v = max(v, dpp(v, integral_constant<int, 0xB1>{}));
    v = max(v, dpp(v, integral_constant<int, 0x4E>{}));
    v = max(v, dpp(v, integral_constant<int, 0x141>{}));
    v = max(v, dpp(v, integral_constant<int, 0x140>{}));
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(uint32_t(p[0]), uint32_t(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(uint32_t(q[0]), uint32_t(q[1]));
}

constexpr double kTopM = 16129.0, kTopV = 4228250625.0;    // 127^2, 255^4
constexpr double kUnitM = 1.0 / kTopM, kUnitV = 1.0 / kTopV;

// code of x in [0, 127^2] (or a hair above: the scale is rounded)
__device__ __forceinline__ int exact_level2(double x, uint32_t u)
{
    int c = int(sqrtf(float(x)));
    c -= double(c * c) > x;
    c += double((c + 1) * (c + 1)) <= x;
    const bool up = (x - double(c * c)) * 65536.0 > double(u * uint32_t(2 * c + 1));
    return min(c + int(up), 127);
}
// code of x in [0, 255^4]
__device__ __forceinline__ int exact_level4(double x, uint32_t u)
{
    const auto four = [](int c) {
        const uint32_t s = uint32_t(c * c);
        return double(s) * double(s);
    };
    int c = min(int(sqrtf(sqrtf(float(x)))), 255);
    c -= four(c) > x;
    c += four(c + 1) <= x;
    const double lo = four(c);
    const bool up = (x - lo) * 65536.0 > double(u) * (four(c + 1) - lo);
    return min(c + int(up), 255);
}

// The same in fp32: the level, and in `least` the least of what decides it less the error
// of that (of 65536 times the value's share of its interval, `width` wide, against u).
// x is within 3 roundings and a reciprocal's ulp (3e-7 of it) of the exact one, so the
// error is less than 2 of u's steps. Next to an end of the interval the exact x may lie in
// the next one, or c be that one's for the square roots' ulps (of x: 2.4e-7 for m, 7.2e-7
// for v's two): up to 1.02e-6 x / width <= 6.5e-5 of the interval, 4.3 steps, and both
// decide alike unless u is within 5 of its own ends; within 6 is left to fp64 (one wave in
// eleven has some).
__device__ __forceinline__ float level2(float x, float u, float &least)
{
    const float c = floorf(__builtin_amdgcn_sqrtf(x));
    const float d = __builtin_fmaf(-c, c, x), width = __builtin_fmaf(2.f, c, 1.f);
    const float over = d * 65536.f - u * width;                  // the product is exact
    least = fminf(least, fabsf(over) - x * (3.6e-7f * 65536.f));
    return fminf(c + (over > 0.f ? 1.f : 0.f), 127.f);
}
__device__ __forceinline__ float level4(float x, float u, float &least)
{
    const float c = fminf(floorf(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(x))), 255.f), s = c * c;
    const float d = __builtin_fmaf(-s, s, x);
    const float width = __builtin_fmaf(c, __builtin_fmaf(c, __builtin_fmaf(c, 4.f, 6.f), 4.f), 1.f);
    const float rhs = u * width, over = d * 65536.f - rhs;
    least = fminf(least, fabsf(over) - (x * (4.2e-7f * 65536.f) + rhs * 3e-7f));
    return fminf(c + (over > 0.f ? 1.f : 0.f), 255.f);
}

__device__ __forceinline__ double value2(int k, double unit)
{
    const float f = float(k);
    return double(f * fabsf(f)) * unit;        // the square is exact
}
__device__ __forceinline__ double value4(uint32_t k, double unit)
{
    const float f = float(k);
    const double s = double(f * f);
    return s * s * unit;
}

// A lane's elements of the chunk that begins at element `first` of a tensor; WHOLE: all of
// them exist, in all of the workgroup's lanes
template <int BITS, bool WHOLE, typename P, typename G>
__device__ __forceinline__ void adamw_elements(const AdamArgs &a, const AdamTensor &t, int64_t first, int64_t step,
                                               float gs, const float4 &f)
{
    constexpr int kLane = kLaneOf<BITS>;
    const uint32_t i = threadIdx.x * kLane;
    P *const pp = static_cast<P *>(t.p) + first;
    const G *const pg = static_cast<const G *>(t.g) + first;
    const int left = WHOLE ? kLane : int(max(min(t.n - first, adam_chunk(BITS)) - int64_t(i), int64_t(0)));
    float p[kLane], g[kLane], m[kLane], v[kLane];
    Raw<P, kLane> rp;
    Raw<G, kLane> rg;
    if constexpr (WHOLE) {
        rp = load_raw<P, kLane>(pp + i);
        rg = load_raw<G, kLane>(pg + i);
    } else {
        load_some<kLane>(pp + i, left, p);
        load_some<kLane>(pg + i, left, g);
    }
    const auto unpack = [&] {
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            if (WHOLE) {
                p[e] = element(rp, e);
                g[e] = element(rg, e);
            }
            g[e] *= gs;
        }
    };
    if constexpr (BITS == 32) {
        float *pm = static_cast<float *>(t.m) + first, *pv = static_cast<float *>(t.v) + first;
        load_some<kLane>(pm + i, left, m);
        load_some<kLane>(pv + i, left, v);
        unpack();
        const float b1 = float(a.beta1), b2 = float(a.beta2), r1 = float(1.0 - a.beta1), r2 = float(1.0 - a.beta2);
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            m[e] = b1 * m[e] + r1 * g[e];
            v[e] = b2 * v[e] + r2 * (g[e] * g[e]);
        }
        store_some<kLane>(pm + i, left, m);
        store_some<kLane>(pv + i, left, v);
    } else {
        // codes and scales; lanes past the tensor's end hold zeros, whole blocks past it
        // have no scale
        int8_t *pm = static_cast<int8_t *>(t.m) + first;
        uint8_t *pv = static_cast<uint8_t *>(t.v) + first;
        const bool any = WHOLE || first + i / 256 * 256 < t.n;
        float *const ps = t.ms + first / 256, *const pz = t.vs + first / 256;
        float sm = 0.f, sv = 0.f;
        if (any) {
            sm = ps[i / 256];
            sv = pz[i / 256];
        }
        uint32_t cm = 0, cv = 0;
        if (WHOLE || left >= kLane) {
            cm = *reinterpret_cast<const uint32_t *>(pm + i);
            cv = *reinterpret_cast<const uint32_t *>(pv + i);
        } else {
            for (int e = 0; e < left; ++e) {
                cm |= uint32_t(uint8_t(pm[i + e])) << (8 * e);
                cv |= uint32_t(pv[i + e]) << (8 * e);
            }
        }
        // the numbers while the loads are on their way
        const uint4 word = philox(uint64_t(t.first + first) / 4 + threadIdx.x, uint64_t(step), a.seed);
        const uint32_t w[kLane] = {word.x, word.y, word.z, word.w};
        unpack();
        const double um = a.beta1 * (double(sm) * kUnitM), uv = a.beta2 * (double(sv) * kUnitV);
        const double r1 = 1.0 - a.beta1, r2 = 1.0 - a.beta2;
        double md[kLane], vd[kLane];
        uint32_t tm = 0, tv = 0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const bool in = WHOLE || e < left;
            const double gd = double(g[e]);
            md[e] = value2(int(int8_t(cm >> (8 * e))), um) + r1 * gd;
            vd[e] = value4(uint8_t(cv >> (8 * e)), uv) + r2 * (gd * gd);
            if (!in) md[e] = vd[e] = 0.0;
            m[e] = float(md[e]);
            v[e] = float(vd[e]);
            tm = max(tm, __float_as_uint(m[e]) & 0x7fffffffu);
            tv = max(tv, __float_as_uint(v[e]));       // never negative
        }
        tm = wave_max(tm);
        tv = wave_max(tv);
        constexpr uint32_t INF = 0x7f800000u;
        cm = cv = 0;
        if (tm >= INF || tv >= INF) {
            sm = sv = __uint_as_float(0x7fc00000u);
        } else {
            sm = __uint_as_float(tm);
            sv = __uint_as_float(tv);
            const float fm = sm > 0.f ? float(kTopM) * __builtin_amdgcn_rcpf(sm) : 0.f;
            const float fv = sv > 0.f ? float(kTopV) * __builtin_amdgcn_rcpf(sv) : 0.f;
            float km[kLane], kv[kLane], least = 1.f;
            uint32_t lowest = 65535, highest = 0;
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const uint32_t um16 = w[e] & 0xffffu, uv16 = w[e] >> 16;
                km[e] = level2(fabsf(m[e]) * fm, float(um16), least);
                kv[e] = level4(v[e] * fv, float(uv16), least);
                lowest = min(lowest, min(um16, uv16));
                highest = max(highest, max(um16, uv16));
            }
            // A scale so small that its reciprocal leaves fp32, or the scale its normal
            // numbers, is fp64's affair; so is one whose reciprocal is no normal number (above
            // 2^126), for the hardware's is 0 then.
            const auto apart = [](float scale, float least_scale) {
                return scale > 0.f && !(scale > least_scale && scale < 8e37f);
            };
            if (!(least > 0.f) || lowest < 6 || highest > 65529 || apart(sm, 1e-30f) || apart(sv, 1e-26f)) {
                const double xm = sm > 0.f ? kTopM / double(sm) : 0.0, xv = sv > 0.f ? kTopV / double(sv) : 0.0;
#pragma unroll
                for (int e = 0; e < kLane; ++e) {
                    km[e] = float(exact_level2(fabs(md[e]) * xm, w[e] & 0xffffu));
                    kv[e] = float(exact_level4(vd[e] * xv, w[e] >> 16));
                }
            }
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                cm |= (uint32_t(int(copysignf(km[e], m[e]))) & 0xffu) << (8 * e);
                cv |= uint32_t(vd[e] > 0.0 ? fmaxf(kv[e], 1.f) : 0.f) << (8 * e);
            }
        }
        if (WHOLE || left >= kLane) {
            *reinterpret_cast<uint32_t *>(pm + i) = cm;
            *reinterpret_cast<uint32_t *>(pv + i) = cv;
        } else {
            for (int e = 0; e < left; ++e) {
                pm[i + e] = int8_t(cm >> (8 * e));
                pv[i + e] = uint8_t(cv >> (8 * e));
            }
        }
        if (any && (threadIdx.x & 63) == 0) {
            ps[i / 256] = sm;
            pz[i / 256] = sv;
        }
    }
    // With 8 bits the arithmetic is what a step waits for: the hardware's square root and
    // reciprocal, an ulp off each (150 cycles of a SIMD less per element than whole ones),
    // unless a denormal v counts, which that root takes for 0: its term is at most 2^-63 root,
    // and more than eps 2^-24 of the denominator where eps is below 1.8e-12 root.
    float step_of[kLane];
    if (BITS == 8 && f.w > 2e-12f * f.z) {
#pragma unroll
        for (int e = 0; e < kLane; ++e)
            step_of[e] = f.y * m[e] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[e]) * f.z + f.w);
    } else {
#pragma unroll
        for (int e = 0; e < kLane; ++e) step_of[e] = f.y * m[e] / (sqrtf(v[e]) * f.z + f.w);
    }
    // (p times 1 - lr weight_decay would take that factor's rounding, 2^-25, for the decay's
    // own: 1.3 % of one of 10^-6, the same way at every step. An infinite p stays so: its decay
    // is the largest finite number's.)
    constexpr float kMost = 3.402823466e38f;
#pragma unroll
    for (int e = 0; e < kLane; ++e)
        p[e] -= __builtin_fmaf(f.x, __builtin_amdgcn_fmed3f(p[e], -kMost, kMost), step_of[e]);
    store_some<kLane>(pp + i, left, p);
    if (t.copy)
        with_type(t.ct, [&](auto z) { store_some<kLane>(static_cast<decltype(z) *>(t.copy) + first + i, left, p); });
}

template <int BITS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamArgs a)
{
    // the tensor of this chunk
    int k = 0;
    while (int(blockIdx.x) >= a.t[k].end) ++k;
    const AdamTensor &t = a.t[k];
    const int64_t first = (int64_t(blockIdx.x) - (k ? a.t[k - 1].end : 0)) * adam_chunk(BITS);
    int64_t step = a.step;
    double rate = a.rate;
    float root = a.root;
    if (a.step_ptr) {
        // by one lane: 1 - beta^t takes as long as the rest of the step
        __shared__ double factor[2];
        step = *a.step_ptr;
        if (threadIdx.x == 0) {
            factor[0] = 1.0 / correction(a.beta1, step);
            factor[1] = 1.0 / sqrt(correction(a.beta2, step));
        }
        __syncthreads();
        rate = factor[0];
        root = float(factor[1]);
    }
    const float lr = t.lr * (a.lr_ptr ? *a.lr_ptr : 1.f), gs = a.grad_scale * (a.grad_scale_ptr ? *a.grad_scale_ptr : 1.f);
    // p - (decay p + rate m / (sqrt(v) root + eps))
    const float4 f{float(double(lr) * double(t.decay)), float(double(lr) * rate), root, a.eps};
    with_type(t.pt, [&](auto p) {
        with_type(t.gt, [&](auto g) {
            if (first + adam_chunk(BITS) <= t.n)
                adamw_elements<BITS, true, decltype(p), decltype(g)>(a, t, first, step, gs, f);
            else
                adamw_elements<BITS, false, decltype(p), decltype(g)>(a, t, first, step, gs, f);
        });
    });
}

// 4 elements a lane: a wave's loads and stores are consecutive
__global__ __launch_bounds__(kThreads) void adamw_values_kernel(int64_t n, const int8_t *m, const uint8_t *v,
                                                                const float *ms, const float *vs, float *mo, float *vo)
{
    const int64_t step = int64_t(gridDim.x) * kThreads * 4;
    for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 4; i < n; i += step) {
        const int64_t left = n - i;
        const double um = double(ms[i / 256]) / kTopM, uv = double(vs[i / 256]) / kTopV;
        uint32_t cm = 0, cv = 0;
        if (left >= 4) {
            cm = *reinterpret_cast<const uint32_t *>(m + i);
            cv = *reinterpret_cast<const uint32_t *>(v + i);
        } else {
            for (int e = 0; e < left; ++e) {
                cm |= uint32_t(uint8_t(m[i + e])) << (8 * e);
                cv |= uint32_t(v[i + e]) << (8 * e);
            }
        }
        float a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = float(value2(int(int8_t(cm >> (8 * e))), um));
            b[e] = float(value4(uint8_t(cv >> (8 * e)), uv));
        }
        store_some<4>(mo + i, left, a);
        store_some<4>(vo + i, left, b);
    }
}

}  // namespace

hipError_t launch_adamw(const AdamArgs &a, int bits, hipStream_t s)
{
    const dim3 grid(unsigned(a.t[a.count - 1].end));
    if (bits == 8)
        hipLaunchKernelGGL((adamw_kernel<8>), grid, dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((adamw_kernel<32>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_adamw_values(int64_t n, const void *m, const void *v, const float *ms, const float *vs, float *mo,
                               float *vo, hipStream_t s)
{
    const int64_t groups = std::min<int64_t>((n + kThreads * 4 - 1) / (kThreads * 4), int64_t(1) << 20);
    hipLaunchKernelGGL(adamw_values_kernel, dim3(unsigned(groups)), dim3(kThreads), 0, s, n,
                       static_cast<const int8_t *>(m), static_cast<const uint8_t *>(v), ms, vs, mo, vo);
    return hipGetLastError();
}

}  // namespace im2win
