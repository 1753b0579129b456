// Layer norm over the channels of NCHW feature maps: forward and backward.
// Bound by HBM like the row kernels; here a position's channels are P elements
// apart, so a workgroup takes a tile of 64 consecutive positions of one image
// and all its channels. Thread (g, l) holds positions 4l .. 4l+3 (one vector
// load per channel, 16 lanes reading consecutive memory) of channels g, g + 32,
// ...; the sums over the channels go through LDS. Backward, a thread's share
// of dweight and dbias stays in registers over all tiles the workgroup takes.
// Maps of more than 32 * 16 channels are read again for each pass.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm_common.hpp"

namespace im2win {
namespace {

constexpr int kPosLanes = 16, kPos = 64, kChanGroups = 32, kThreads = kPosLanes * kChanGroups;

// per position, the sum over the channel groups
__device__ __forceinline__ void chan_sum(float (&v)[4], float (*red)[kPos])
{
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes;
    // a wave holds 4 channel groups: add those first
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] += __shfl_xor(v[e], 16, 64);
        v[e] += __shfl_xor(v[e], 32, 64);
    }
    __syncthreads();
    if ((g & 3) == 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[g >> 2][l * 4 + e] = v[e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < kChanGroups / 4; ++q) t += red[q][l * 4 + e];
        v[e] = t;
    }
}

// KR: channels per thread held in registers; 0: any number, read again for
// each pass
template <typename TX, typename TY, int KR>
__global__ __launch_bounds__(kThreads) void norm_nchw_fwd_kernel(const NormArgs a, int tiles_p)
{
    __shared__ float red[kChanGroups / 4][kPos];
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes, C = a.C;
    const float fc = float(C);
    const int64_t tiles = a.N * tiles_p;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t n = t / tiles_p, p = (t - n * tiles_p) * kPos + l * 4;
        const int left = int(min(int64_t(4), a.P - p));           // <= 0: no position here
        const int64_t base = n * C * a.P + p;
        const TX *x = static_cast<const TX *>(a.x) + base;
        TY *y = static_cast<TY *>(a.out) + base;
        float v[KR ? KR : 1][4], mean[4] = {}, var[4] = {};
        auto each = [&](auto f) {
            if constexpr (KR > 0) {
#pragma unroll
                for (int i = 0; i < KR; ++i) {
                    const int c = g + i * kChanGroups;
                    if (c < C) f(c, v[i]);
                }
            } else {
                for (int c = g; c < C; c += kChanGroups) {
                    load_some<4>(x + c * a.P, left, v[0]);
                    f(c, v[0]);
                }
            }
        };
        if constexpr (KR > 0) each([&](int c, float (&u)[4]) { load_some<4>(x + c * a.P, left, u); });
        each([&](int, float (&u)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) mean[e] += u[e];
        });
        chan_sum(mean, red);
#pragma unroll
        for (int e = 0; e < 4; ++e) mean[e] /= fc;
        each([&](int, float (&u)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) var[e] += (u[e] - mean[e]) * (u[e] - mean[e]);
        });
        chan_sum(var, red);
        float rstd[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) rstd[e] = 1.f / sqrtf(var[e] / fc + a.eps);
        if (g == 0 && a.mean) {
            store_some<4>(a.mean + n * a.P + p, left, mean);
            store_some<4>(a.rstd + n * a.P + p, left, rstd);
        }
        if (left > 0)
            each([&](int c, float (&u)[4]) {
                const float w = a.weight ? a.weight[c] : 1.f, b = a.bias ? a.bias[c] : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = (u[e] - mean[e]) * rstd[e] * w + b;
                if (a.drop.threshold) drop_run<4>(base + c * a.P, a.drop, u);
                store_some<4>(y + c * a.P, left, u);
            });
    }
}

template <typename TX, typename TY, int KR>
__global__ __launch_bounds__(kThreads) void norm_nchw_bwd_kernel(const NormArgs a, int tiles_p)
{
    constexpr int KA = KR ? KR : 1;
    __shared__ float red[kChanGroups / 4][kPos];
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes, C = a.C;
    const float fc = float(C);
    const int64_t tiles = a.N * tiles_p;
    float dw[KA], db[KA];
#pragma unroll
    for (int i = 0; i < KA; ++i) dw[i] = db[i] = 0.f;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t n = t / tiles_p, p = (t - n * tiles_p) * kPos + l * 4;
        const int left = int(min(int64_t(4), a.P - p));
        const int64_t base = n * C * a.P + p;
        const TX *x = static_cast<const TX *>(a.x) + base;
        const TY *dy = static_cast<const TY *>(a.dy) + base;
        TX *dx = static_cast<TX *>(a.out) + base;
        float mean[4], rstd[4], s1[4] = {}, s2[4] = {};
        load_some<4>(a.mean + n * a.P + p, left, mean);
        load_some<4>(a.rstd + n * a.P + p, left, rstd);
        float h[KA][4], z[KA][4];
        auto load = [&](int c, float (&hc)[4], float (&zc)[4]) {       // xhat and dz
            load_some<4>(x + c * a.P, left, hc);
            load_some<4>(dy + c * a.P, left, zc);
            if (a.drop.threshold && left > 0) drop_run<4>(base + c * a.P, a.drop, zc);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hc[e] = e < left ? (hc[e] - mean[e]) * rstd[e] : 0.f;
                zc[e] = e < left ? zc[e] : 0.f;
            }
        };
        auto each = [&](auto f) {
            if constexpr (KR > 0) {
#pragma unroll
                for (int i = 0; i < KR; ++i) {
                    const int c = g + i * kChanGroups;
                    if (c < C) f(i, c, h[i], z[i]);
                }
            } else {
                for (int c = g; c < C; c += kChanGroups) {
                    load(c, h[0], z[0]);
                    f(0, c, h[0], z[0]);
                }
            }
        };
        if constexpr (KR > 0) each([&](int, int c, float (&hc)[4], float (&zc)[4]) { load(c, hc, zc); });
        each([&](int i, int c, float (&hc)[4], float (&zc)[4]) {
            const float w = a.weight ? a.weight[c] : 1.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (KR > 0) {
                    dw[i] += zc[e] * hc[e];
                    db[i] += zc[e];
                }
                s1[e] += zc[e] * w;
                s2[e] += zc[e] * w * hc[e];
            }
        });
        chan_sum(s1, red);
        chan_sum(s2, red);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s1[e] /= fc;
            s2[e] /= fc;
        }
        if (left > 0)
            each([&](int, int c, float (&hc)[4], float (&zc)[4]) {
                const float w = a.weight ? a.weight[c] : 1.f;
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = rstd[e] * (zc[e] * w - s1[e] - hc[e] * s2[e]);
                store_some<4>(dx + c * a.P, left, o);
            });
    }
    if constexpr (KR > 0) {
        if (!a.partial) return;
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const float u = lane_sum<kPosLanes>(dw[i]), v = lane_sum<kPosLanes>(db[i]);
            const int c = g + i * kChanGroups;
            if (l == 0 && c < C) {
                a.partial[(int64_t(blockIdx.x) * 2 + 0) * C + c] = u;
                a.partial[(int64_t(blockIdx.x) * 2 + 1) * C + c] = v;
            }
        }
    }
}

// weight gradients of maps read again for each pass: a wave takes one channel
// of every gridDim.y-th image
template <typename TX, typename TY>
__global__ __launch_bounds__(256) void norm_planes_kernel(const NormArgs a)
{
    const int c = blockIdx.x * 4 + (threadIdx.x >> 6), l = threadIdx.x & 63, C = a.C;
    if (c >= C) return;
    float dw = 0.f, db = 0.f;
    for (int64_t n = blockIdx.y; n < a.N; n += gridDim.y) {
        const int64_t base = (n * C + c) * a.P;
        for (int64_t p = l * 4; p < a.P; p += 256) {
            const int left = int(min(int64_t(4), a.P - p));
            float h[4], z[4], mean[4], rstd[4];
            load_some<4>(static_cast<const TX *>(a.x) + base + p, left, h);
            load_some<4>(static_cast<const TY *>(a.dy) + base + p, left, z);
            load_some<4>(a.mean + n * a.P + p, left, mean);
            load_some<4>(a.rstd + n * a.P + p, left, rstd);
            if (a.drop.threshold) drop_run<4>(base + p, a.drop, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dw += e < left ? z[e] * (h[e] - mean[e]) * rstd[e] : 0.f;
                db += e < left ? z[e] : 0.f;
            }
        }
    }
    dw = lane_sum<64>(dw);
    db = lane_sum<64>(db);
    if (l == 0) {
        a.partial[(int64_t(blockIdx.y) * 2 + 0) * C + c] = dw;
        a.partial[(int64_t(blockIdx.y) * 2 + 1) * C + c] = db;
    }
}

// channels per thread held in registers (0: too many)
int regs_of(int64_t C)
{
    for (int k : {2, 4, 8, 16})
        if (C <= int64_t(k) * kChanGroups) return k;
    return 0;
}

template <typename F>
hipError_t with_regs(int kr, F f)
{
    using std::integral_constant;
    switch (kr) {
    case 2: return f(integral_constant<int, 2>{});
    case 4: return f(integral_constant<int, 4>{});
    case 8: return f(integral_constant<int, 8>{});
    case 16: return f(integral_constant<int, 16>{});
    default: return f(integral_constant<int, 0>{});
    }
}

constexpr int64_t kMaxBlocksFwd = 2048, kMaxBlocksBwd = 512, kImageSplits = 16;

int64_t tiles_of(int64_t N, int64_t P) { return N * ((P + kPos - 1) / kPos); }

}  // namespace

int64_t norm_nchw_partials(int64_t N, int64_t C, int64_t P)
{
    if (!regs_of(C)) return kImageSplits;
    return std::max<int64_t>(1, std::min(tiles_of(N, P), kMaxBlocksBwd));
}

hipError_t launch_norm_nchw_fwd(const NormArgs &a, hipStream_t s)
{
    const int64_t tiles = tiles_of(a.N, a.P);
    const dim3 grid(unsigned(std::min(tiles, kMaxBlocksFwd)));
    const int tiles_p = int((a.P + kPos - 1) / kPos);
    return with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        return with_regs(regs_of(a.C), [&](auto kr) {
            hipLaunchKernelGGL((norm_nchw_fwd_kernel<typename decltype(tx)::type, typename decltype(ty)::type,
                                                     decltype(kr)::value>),
                               grid, dim3(kThreads), 0, s, a, tiles_p);
            return hipGetLastError();
        });
    });
}

hipError_t launch_norm_nchw_bwd(const NormArgs &a, hipStream_t s)
{
    const int64_t blocks = norm_nchw_partials(a.N, a.C, a.P);
    const int tiles_p = int((a.P + kPos - 1) / kPos), kr = regs_of(a.C);
    hipError_t e = with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        const dim3 grid(unsigned(kr ? blocks
                                    : std::max<int64_t>(1, std::min(tiles_of(a.N, a.P), kMaxBlocksFwd))));
        hipError_t e1 = with_regs(kr, [&](auto k) {
            hipLaunchKernelGGL((norm_nchw_bwd_kernel<TX, TY, decltype(k)::value>), grid, dim3(kThreads), 0, s, a,
                               tiles_p);
            return hipGetLastError();
        });
        if (e1 != hipSuccess || kr || !a.partial) return e1;
        hipLaunchKernelGGL((norm_planes_kernel<TX, TY>), dim3(unsigned((a.C + 3) / 4), unsigned(blocks)),
                           dim3(256), 0, s, a);
        return hipGetLastError();
    });
    if (e != hipSuccess || !a.partial) return e;
    return launch_norm_reduce(a.partial, blocks, a.C, a.dweight, a.dbias, s);
}

}  // namespace im2win
