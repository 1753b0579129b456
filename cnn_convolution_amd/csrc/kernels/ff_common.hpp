// Shared by the feed-forward kernels: the activations, the scale of fp16 gradients.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../ff.hpp"
#include "im2win_block.h"

namespace im2win {

// 1 / (1 + exp(-a)): fp32 outputs keep their digits (expf and the division are within
// an ulp or two); half precision takes the hardware's exp2 and reciprocal, a few fp32
// ulp off, which is all that the epilogue of a 256 x 256 tile has time for
template <bool EXACT>
__device__ __forceinline__ float logistic(float a)
{
    if constexpr (EXACT) return 1.f / (1.f + expf(-a));
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(a * -1.4426950408889634f));
}

// act(a) and its slope. EXACT: for fp32 outputs.
template <bool EXACT>
__device__ __forceinline__ void activate(int act, float a, float &f, float &df)
{
    if (act == FF_SILU) {
        const float s = logistic<EXACT>(a);
        f = a * s;
        df = s * (1.f + a * (1.f - s));
    } else if (act == FF_SIGMOID) {
        // the smaller of f and 1 - f from the exponential: 1 - f by itself has no digits
        // left where f is next to 1
        const float x = fabsf(a), e = EXACT ? expf(-x) : __builtin_amdgcn_exp2f(x * -1.4426950408889634f);
        const float r = EXACT ? 1.f / (1.f + e) : __builtin_amdgcn_rcpf(1.f + e);
        f = a < 0.f ? e * r : r;
        df = e * r * r;
    } else if (act == FF_GELU) {
        if constexpr (EXACT) {
            const float c = 0.5f * erfcf(a * -0.70710678118654752f);   // (1 + erf has no digits left below -5)
            f = a * c;
            df = c + a * (expf(-0.5f * a * a) * 0.39894228040143268f);
        } else {
            // erfc(z) exp(z^2) as a polynomial of t = 1 / (1 + 0.33 z), fitted here (least
            // squares with weights moved to the largest relative error, z up to 10): within
            // 1e-7 of itself, so that act(a) keeps its digits where erfc is small. The
            // exponential is the slope's too (erff and another made a third of the gate's
            // launch: 4097 x 1032 x 3001, fp16, 120 us).
            const float z = fabsf(a) * 0.70710678118654752f, e = __builtin_amdgcn_exp2f(z * z * -1.4426950408889634f);
            const float t = __builtin_amdgcn_rcpf(1.f + 0.33f * z);
            const float c4 = 0.408491522f + t * (-0.351140231f + t * (0.460231423f + t * -0.135344267f));
            const float q = t * (0.186357796f + t * (0.182956144f + t * (0.201222599f + t * (0.0472249985f + t * c4))));
            const float lower = 0.5f * q * e, c = a < 0.f ? lower : 1.f - lower;
            f = a * c;
            df = c + a * (e * 0.39894228040143268f);
        }
    } else if (act == FF_GELU_TANH) {
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)); beyond 100 it is 0 or 1 whatever a^2 is,
        // which must not be infinite beside the 0 in the slope
        const float k = 1.5957691216057308f, q = 0.044715f * fminf(a * a, 1e4f);
        const float s = logistic<EXACT>(k * a * (1.f + q));
        f = a * s;
        df = s + a * s * (1.f - s) * k * (1.f + 3.f * q);
    } else {
        f = a < 0.f ? 0.f : a;               // NaN stays
        df = a > 0.f ? 1.f : 0.f;
    }
}

// fp16's da and du are held times S, a power of two for each row with S * max |dy| of the
// row in [2^-4, 2^-3), which dx takes back: no row's dx depends on another row. They may be
// 2^19 times that maximum before they are infinite, and down to 2^-10 of it keep all digits;
// a smaller one is off by at most 2^-21 of it. The weights' gradients are sums over the rows:
// they read x times M / S, with one M for all rows, the least S times the power of two that
// brings the largest |x| into [2^6, 2^7), so that a row whose dy is 2^-10 of the largest
// still has x down to 2^-10 of the largest with all digits. x so scaled is written by
// workgroups of the back launch: 8192 x 2048 x 8192 390 us for 375 (with da and du written
// twice instead, times S and times the least S, 507).
// Rows of zeros have S 2^100: neither their x nor its size is anything to the others.
__device__ __forceinline__ float scale_of(float m)
{
    if (!(m > 0.f)) return 1.f;
    int e = 0;
    (void)frexpf(m, &e);                     // m = f 2^e, f in [1/2, 1)
    return ldexpf(1.f, -3 - e);
}
constexpr float kZeroRow = 1.2676506002282294e30f;           // 2^100

// of kAmaxParts maxima, by every wave for itself
__device__ __forceinline__ float scale_of_parts(const float *amax)
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kAmaxParts / 64; ++i) m = fmaxf(m, amax[(threadIdx.x & 63) + i * 64]);
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
    return scale_of(m);
}
// the least S, and what brings x into its range
__device__ __forceinline__ float dy_scale(const float *amax) { return scale_of_parts(amax); }
__device__ __forceinline__ float x_scale(const float *amax) { return scale_of_parts(amax + kAmaxParts) * 1024.f; }

template <typename F>
hipError_t with_ff_type(int dtype, F f)
{
    if (dtype == 0) return f(float{});
    if (dtype == 1) return f(_Float16{});
    return f(__bf16{});
}

}  // namespace im2win
