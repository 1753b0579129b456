// One AdamW step over many tensors (im2win_block.h), states in 32 or in 8 bits, and
// the values of 8-bit states. Bound by HBM: every element of p, g, m and v is read and
// of p, m and v written once.
//
// A launch takes up to kAdamTensors tensors by value, a workgroup one chunk of 2048
// consecutive elements of one of them, a lane 8 consecutive ones: half a wave holds a
// block of 256 of an 8-bit state, whose scale is a maximum over 32 lanes, so the states
// need one pass and no LDS. The types of p, g and copy are a workgroup's affair (a
// branch that all its lanes take alike).
//
// 8-bit states are formed in fp64, where the level that an element gets, and so the
// step, is the definition's to the last bit whatever the order of operations: a value in
// units of its block's scale, x = |m| 127^2 / M or v 255^4 / V, lies between c^2 (c^4) and
// (c + 1)^2 ((c + 1)^4), all whole numbers below 2^53; c comes from fp32 square roots
// and is put right by comparing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../block_launch.hpp"
#include "head_vec.hpp"
#include "philox.hpp"

namespace im2win {
namespace {

constexpr int kThreads = 256;
constexpr int kLane = 8;                       // elements of a lane
static_assert(kThreads * kLane == kAdamChunk, "one round per chunk");

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

// the step's factors, the same for all elements of a tensor
struct Factors {
    float keep, rate, root, eps;               // p keep - rate m / (sqrt(v) root + eps)
};

// 1 - beta^t in fp64; beta 0: 1
__device__ __forceinline__ double correction(double beta, int64_t t)
{
    return beta > 0.0 ? -expm1(double(t) * log(beta)) : 1.0;
}

// largest |value| of an aligned half wave as bits: NaN and infinity are above all
__device__ __forceinline__ uint32_t half_wave_max(uint32_t v)
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
    return max(uint32_t(p[0]), uint32_t(p[1]));
}

constexpr double kTopM = 16129.0, kTopV = 4228250625.0;    // 127^2, 255^4

// code of x in [0, 127^2] (with a hair above: the scale is rounded)
__device__ __forceinline__ int level2(double x, uint32_t u)
{
    int c = int(sqrtf(float(x)));
    c -= double(c * c) > x;
    c += double((c + 1) * (c + 1)) <= x;
    const bool up = (x - double(c * c)) * 65536.0 > double(u * uint32_t(2 * c + 1));
    return min(c + int(up), 127);
}
// code of x in [0, 255^4]
__device__ __forceinline__ int level4(double x, uint32_t u)
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

__device__ __forceinline__ double value2(int k, double unit) { return double(k * abs(k)) * unit; }
__device__ __forceinline__ double value4(int k, double unit)
{
    const double s = double(k * k);
    return s * s * unit;
}

template <int BITS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamArgs a)
{
    // the tensor of this chunk
    int k = 0;
    while (int(blockIdx.x) >= a.t[k].end) ++k;
    const AdamTensor &t = a.t[k];
    const int64_t chunk = int64_t(blockIdx.x) - (k ? a.t[k - 1].end : 0);
    const int64_t i = chunk * kAdamChunk + threadIdx.x * kLane, left = t.n - i;

    __shared__ Factors shared;
    const int64_t step = a.step_ptr ? *a.step_ptr : a.step;
    if (threadIdx.x == 0) {
        const float lr = t.lr * (a.lr_ptr ? *a.lr_ptr : 1.f);
        const double c1 = correction(a.beta1, step), c2 = correction(a.beta2, step);
        shared = Factors{float(1.0 - double(lr) * double(t.decay)), float(double(lr) / c1), float(1.0 / sqrt(c2)), a.eps};
    }
    const float gs = a.grad_scale * (a.grad_scale_ptr ? *a.grad_scale_ptr : 1.f);

    float p[kLane], g[kLane], m[kLane], v[kLane];
    with_type(t.pt, [&](auto z) { load_some<kLane>(static_cast<const decltype(z) *>(t.p) + i, max(left, int64_t(0)), p); });
    with_type(t.gt, [&](auto z) { load_some<kLane>(static_cast<const decltype(z) *>(t.g) + i, max(left, int64_t(0)), g); });
#pragma unroll
    for (int e = 0; e < kLane; ++e) g[e] *= gs;

    if constexpr (BITS == 32) {
        float *pm = static_cast<float *>(t.m) + i, *pv = static_cast<float *>(t.v) + i;
        load_some<kLane>(pm, max(left, int64_t(0)), m);
        load_some<kLane>(pv, max(left, int64_t(0)), v);
        const float b1 = float(a.beta1), b2 = float(a.beta2), r1 = float(1.0 - a.beta1), r2 = float(1.0 - a.beta2);
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            m[e] = b1 * m[e] + r1 * g[e];
            v[e] = b2 * v[e] + r2 * (g[e] * g[e]);
        }
        store_some<kLane>(pm, max(left, int64_t(0)), m);
        store_some<kLane>(pv, max(left, int64_t(0)), v);
    } else {
        // codes and scales; lanes past the tensor's end hold zeros, whole blocks past it
        // have no scale
        int8_t *pm = static_cast<int8_t *>(t.m) + i;
        uint8_t *pv = static_cast<uint8_t *>(t.v) + i;
        const bool any = i / 256 * 256 < t.n;
        double um = 0.0, uv = 0.0;
        if (any) {
            um = double(t.ms[i / 256]) / kTopM;
            uv = double(t.vs[i / 256]) / kTopV;
        }
        double md[kLane], vd[kLane];
        uint64_t cm = 0, cv = 0;
        if (left >= kLane) {
            cm = *reinterpret_cast<const uint64_t *>(pm);
            cv = *reinterpret_cast<const uint64_t *>(pv);
        } else {
            for (int e = 0; e < left; ++e) {
                cm |= uint64_t(uint8_t(pm[e])) << (8 * e);
                cv |= uint64_t(pv[e]) << (8 * e);
            }
        }
        uint32_t tm = 0, tv = 0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const double gd = double(g[e]);
            md[e] = a.beta1 * value2(int(int8_t(cm >> (8 * e))), um) + (1.0 - a.beta1) * gd;
            vd[e] = a.beta2 * value4(int(uint8_t(cv >> (8 * e))), uv) + (1.0 - a.beta2) * (gd * gd);
            if (e >= left) md[e] = vd[e] = 0.0;
            m[e] = float(md[e]);
            v[e] = float(vd[e]);
            tm = max(tm, __float_as_uint(m[e]) & 0x7fffffffu);
            tv = max(tv, __float_as_uint(v[e]) & 0x7fffffffu);
        }
        tm = half_wave_max(tm);
        tv = half_wave_max(tv);
        constexpr uint32_t INF = 0x7f800000u;
        const bool bad = tm >= INF || tv >= INF;
        const float sm = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(tm);
        const float sv = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(tv);
        const double xm = sm > 0.f ? kTopM / double(sm) : 0.0, xv = sv > 0.f ? kTopV / double(sv) : 0.0;
        const uint64_t block = uint64_t(t.first + i) / 4;
        const uint4 w0 = philox(block, uint64_t(step), a.seed), w1 = philox(block + 1, uint64_t(step), a.seed);
        const uint32_t w[kLane] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        cm = cv = 0;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            int km = bad ? 0 : level2(fabs(md[e]) * xm, w[e] & 0xffffu);
            int kv = bad ? 0 : level4(vd[e] * xv, w[e] >> 16);
            km = md[e] < 0.0 ? -km : km;
            kv = vd[e] > 0.0 && !bad ? max(kv, 1) : 0;
            cm |= uint64_t(uint8_t(km)) << (8 * e);
            cv |= uint64_t(uint8_t(kv)) << (8 * e);
        }
        if (left >= kLane) {
            *reinterpret_cast<uint64_t *>(pm) = cm;
            *reinterpret_cast<uint64_t *>(pv) = cv;
        } else {
            for (int e = 0; e < left; ++e) {
                pm[e] = int8_t(cm >> (8 * e));
                pv[e] = uint8_t(cv >> (8 * e));
            }
        }
        if (any && (threadIdx.x & 31) == 0) {
            t.ms[i / 256] = sm;
            t.vs[i / 256] = sv;
        }
    }
    __syncthreads();
    const Factors f = shared;
#pragma unroll
    for (int e = 0; e < kLane; ++e) p[e] = p[e] * f.keep - f.rate * m[e] / (sqrtf(v[e]) * f.root + f.eps);
    with_type(t.pt, [&](auto z) { store_some<kLane>(static_cast<decltype(z) *>(t.p) + i, max(left, int64_t(0)), p); });
    if (t.copy)
        with_type(t.ct, [&](auto z) { store_some<kLane>(static_cast<decltype(z) *>(t.copy) + i, max(left, int64_t(0)), p); });
}

__global__ __launch_bounds__(kThreads) void adamw_values_kernel(int64_t n, const int8_t *m, const uint8_t *v,
                                                                const float *ms, const float *vs, float *mo, float *vo)
{
    const int64_t step = int64_t(gridDim.x) * kThreads * kLane;
    for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * kLane; i < n; i += step) {
        const int64_t left = n - i;
        const double um = double(ms[i / 256]) / kTopM, uv = double(vs[i / 256]) / kTopV;
        float a[kLane], b[kLane];
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            a[e] = e < left ? float(value2(m[i + e], um)) : 0.f;
            b[e] = e < left ? float(value4(v[i + e], uv)) : 0.f;
        }
        store_some<kLane>(mo + i, left, a);
        store_some<kLane>(vo + i, left, b);
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
    const int64_t groups = std::min<int64_t>((n + kAdamChunk - 1) / kAdamChunk, 8192);
    hipLaunchKernelGGL(adamw_values_kernel, dim3(unsigned(groups)), dim3(kThreads), 0, s, n,
                       static_cast<const int8_t *>(m), static_cast<const uint8_t *>(v), ms, vs, mo, vo);
    return hipGetLastError();
}

}  // namespace im2win
