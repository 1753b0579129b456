// Layer norm over the channels of NCHW feature maps: forward and backward.
// Bound by HBM like the row kernels; here a position's channels are P elements
// apart, so a workgroup takes a tile of 64 consecutive positions of one image
// and all its channels. Thread (g, l) holds positions 4l .. 4l+3 (one vector
// load per channel, 16 lanes reading consecutive memory) of KR channels g, g +
// groups, ...; a wave adds its channels in registers, the waves' sums meet in
// LDS. Backward, a thread's share of dweight and dbias stays in registers over
// all tiles the workgroup takes. Maps of more than 512 channels, or fewer than 4
// positions, are read again for each pass.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm_common.hpp"

namespace im2win {
namespace {

constexpr int kPosLanes = 16, kPos = 64;

// v[e] over the lanes of a wave that hold the same positions
__device__ __forceinline__ void wave_chan_sum(float (&v)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = __float_as_uint(v[e]);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const uint32_t w = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
        const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
        v[e] = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
}

// where this thread's tile lies
struct TilePos {
    int64_t n, p, base;      // image, first position, offset of channel 0 there
    int left;                // positions that exist (<= 0: none)
    __device__ __forceinline__ TilePos(int64_t t, int tiles_p, int l, const NormArgs &a)
    {
        n = t / tiles_p;
        p = (t - n * tiles_p) * kPos + l * 4;
        left = int(min(int64_t(4), a.P - p));
        base = n * a.C * a.P;
    }
};

template <bool EXACT, typename T>
__device__ __forceinline__ void store_pos(T *p, int left, const float (&f)[4])
{
    if constexpr (EXACT) {
        if (left > 0) store_vec<4>(p, f);
    } else {
        store_some<4>(p, left, f);
    }
}

// Elements of an image are addressed as its (wave-uniform) base and a 32-bit
// byte offset per lane: half the registers of a pointer per channel. The images
// these kernels take are below 4 GB.
template <typename T>
__device__ __forceinline__ const T *at_offset(const T *base, uint32_t elems)
{
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(base) + elems * uint32_t(sizeof(T)));
}
template <typename T>
__device__ __forceinline__ T *at_offset(T *base, uint32_t elems)
{
    return reinterpret_cast<T *>(reinterpret_cast<char *>(base) + elems * uint32_t(sizeof(T)));
}

// where positions p .. p + 3 of a channel are read from, and how far that is
// before p (see load_row)
struct Window {
    uint32_t at;
    int shift;
    __device__ __forceinline__ Window(int64_t p, int64_t P)
    {
        const int64_t q = p < P - 4 ? p : P - 4;
        at = uint32_t(q);
        shift = int(p - q < 4 ? p - q : 4);
    }
};

// WAVES waves, 4 * WAVES channel groups; EXACT: P is a multiple of 4
template <typename TX, typename TY, int WAVES, int KR, bool EXACT>
__global__ __launch_bounds__(WAVES * 64) void norm_nchw_fwd_kernel(const NormArgs a, int tiles_p)
{
    constexpr int G = WAVES * 4;
    __shared__ __align__(16) float red[2][WAVES][kPos];    // mean, squares
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes, wave = threadIdx.x >> 6, C = a.C;
    const float fc = float(C);
    const uint32_t P = uint32_t(a.P);
    float w[KR], b[KR];
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        const int c = min(g + i * G, C - 1);
        w[i] = a.weight ? a.weight[c] : 1.f;
        b[i] = a.bias ? a.bias[c] : 0.f;
    }
    // channels that wave q holds
    auto count = [&](int q) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < KR; ++i) n += max(0, min(4, C - i * G - q * 4));
        return float(n);
    };
    const TilePos at(blockIdx.x, tiles_p, l, a);
    const TX *x = static_cast<const TX *>(a.x) + at.base;
    TY *y = static_cast<TY *>(a.out) + at.base;
    const Window win(at.p, a.P);
    // channels past the last read that one and count nowhere
    Raw<TX, 4> q[KR];
#pragma unroll
    for (int i = 0; i < KR; ++i)
        q[i] = load_raw<TX, 4>(at_offset(x, uint32_t(min(g + i * G, C - 1)) * P + win.at));
    if constexpr (!EXACT)
#pragma unroll
        for (int i = 0; i < KR; ++i) shift_down(q[i], win.shift);
    float v[KR][4], mean[4] = {}, sq[4] = {};
#pragma unroll
    for (int i = 0; i < KR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[i][e] = element(q[i], e);
            mean[e] += g + i * G < C ? v[i][e] : 0.f;
        }
    // a wave's own mean and squared deviations, joined with one barrier:
    // sum (x - mean)^2 = sum_w [Q_w + n_w (mean_w - mean)^2]
    wave_chan_sum(mean);
    const float nw = fmaxf(count(wave), 1.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) mean[e] /= nw;
#pragma unroll
    for (int i = 0; i < KR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float d = v[i][e] - mean[e];
            sq[e] += g + i * G < C ? d * d : 0.f;
        }
    wave_chan_sum(sq);
    if ((threadIdx.x & 48) == 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            red[0][wave][l * 4 + e] = mean[e];
            red[1][wave][l * 4 + e] = sq[e];
        }
    __syncthreads();
    float rstd[4], m[4] = {}, s[4] = {};
#pragma unroll 4
    for (int k = 0; k < WAVES; ++k) {
        const float4 u = *reinterpret_cast<const float4 *>(&red[0][k][l * 4]);
        const float n = count(k);
        m[0] += u.x * n;
        m[1] += u.y * n;
        m[2] += u.z * n;
        m[3] += u.w * n;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] /= fc;
#pragma unroll 4
    for (int k = 0; k < WAVES; ++k) {
        const float4 u = *reinterpret_cast<const float4 *>(&red[0][k][l * 4]);
        const float4 q2 = *reinterpret_cast<const float4 *>(&red[1][k][l * 4]);
        const float n = count(k);
        s[0] += q2.x + n * (u.x - m[0]) * (u.x - m[0]);
        s[1] += q2.y + n * (u.y - m[1]) * (u.y - m[1]);
        s[2] += q2.z + n * (u.z - m[2]) * (u.z - m[2]);
        s[3] += q2.w + n * (u.w - m[3]) * (u.w - m[3]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        mean[e] = m[e];
        rstd[e] = 1.f / sqrtf(s[e] / fc + a.eps);
    }
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        const int c = g + i * G;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = (v[i][e] - mean[e]) * rstd[e] * w[i] + b[i];
        if (a.drop.threshold) drop_run<4>(at.base + c * a.P + at.p, a.drop, v[i]);
        store_pos<EXACT>(at_offset(y, c * P + uint32_t(at.p)), c < C ? at.left : 0, v[i]);
    }
    if (g == 0 && a.mean) {
        store_some<4>(a.mean + at.n * a.P + at.p, at.left, mean);
        store_some<4>(a.rstd + at.n * a.P + at.p, at.left, rstd);
    }
}

template <typename TX, typename TY, int WAVES, int KR, bool EXACT>
__global__ __launch_bounds__(WAVES * 64) void norm_nchw_bwd_kernel(const NormArgs a, int tiles_p)
{
    constexpr int G = WAVES * 4;
    __shared__ __align__(16) float red[2][2][WAVES][kPos];
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes, wave = threadIdx.x >> 6, C = a.C;
    const float fc = float(C);
    const int64_t tiles = a.N * tiles_p;
    float w[KR], dw[KR], db[KR];
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        w[i] = a.weight ? a.weight[min(g + i * G, C - 1)] : 1.f;
        dw[i] = db[i] = 0.f;
    }
    int slot = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const TilePos at(t, tiles_p, l, a);
        // opaque, so that no offset of a channel is kept in registers over the tiles
        uint32_t P = uint32_t(a.P);
        asm volatile("" : "+s"(P));
        const TX *x = static_cast<const TX *>(a.x) + at.base;
        const TY *dy = static_cast<const TY *>(a.dy) + at.base;
        TX *dx = static_cast<TX *>(a.out) + at.base;
        const Window win(at.p, a.P);
        const Raw<float, 4> rm = load_row<float, 4, EXACT>(a.mean + at.n * a.P, at.p, a.P);
        const Raw<float, 4> rr = load_row<float, 4, EXACT>(a.rstd + at.n * a.P, at.p, a.P);
        Raw<TX, 4> qx[KR];
        Raw<TY, 4> qy[KR];
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const uint32_t o = uint32_t(min(g + i * G, C - 1)) * P + win.at;
            qx[i] = load_raw<TX, 4>(at_offset(x, o));
            qy[i] = load_raw<TY, 4>(at_offset(dy, o));
        }
        if constexpr (!EXACT)
#pragma unroll
            for (int i = 0; i < KR; ++i) {
                shift_down(qx[i], win.shift);
                shift_down(qy[i], win.shift);
            }
        float h[KR][4], z[KR][4], s1[4] = {}, s2[4] = {};
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const int c = g + i * G;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[i][e] = element(qy[i], e);
            if (a.drop.threshold) drop_run<4>(at.base + uint32_t(c) * P + at.p, a.drop, z[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = c < C && (EXACT ? 0 < at.left : e < at.left);
                h[i][e] = in ? (element(qx[i], e) - element(rm, e)) * element(rr, e) : 0.f;
                z[i][e] = in ? z[i][e] : 0.f;
                dw[i] += z[i][e] * h[i][e];
                db[i] += z[i][e];
                z[i][e] *= w[i];
                s1[e] += z[i][e];
                s2[e] += z[i][e] * h[i][e];
            }
        }
        wave_chan_sum(s1);
        wave_chan_sum(s2);
        if ((threadIdx.x & 48) == 0)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                red[slot][0][wave][l * 4 + e] = s1[e];
                red[slot][1][wave][l * 4 + e] = s2[e];
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) s1[e] = s2[e] = 0.f;
#pragma unroll 4
        for (int k = 0; k < WAVES; ++k) {
            const float4 u = *reinterpret_cast<const float4 *>(&red[slot][0][k][l * 4]);
            const float4 q = *reinterpret_cast<const float4 *>(&red[slot][1][k][l * 4]);
            s1[0] += u.x;
            s1[1] += u.y;
            s1[2] += u.z;
            s1[3] += u.w;
            s2[0] += q.x;
            s2[1] += q.y;
            s2[2] += q.z;
            s2[3] += q.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s1[e] /= fc;
            s2[e] /= fc;
        }
        slot ^= 1;
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const int c = g + i * G;
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = element(rr, e) * (z[i][e] - s1[e] - h[i][e] * s2[e]);
            store_pos<EXACT>(at_offset(dx, c * P + uint32_t(at.p)), c < C ? at.left : 0, o);
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        const float u = lane_sum<kPosLanes>(dw[i]), v = lane_sum<kPosLanes>(db[i]);
        const int c = g + i * G;
        if (l == 0 && c < C) {
            a.partial[(int64_t(blockIdx.x) * 2 + 0) * C + c] = u;
            a.partial[(int64_t(blockIdx.x) * 2 + 1) * C + c] = v;
        }
    }
}

// per position, the sum over the channel groups (for the kernels below)
constexpr int kWide = 512, kWideGroups = kWide / kPosLanes;
__device__ __forceinline__ void chan_sum(float (&v)[4], float (*red)[kPos])
{
    const int l = threadIdx.x % kPosLanes;
    wave_chan_sum(v);
    __syncthreads();
    if ((threadIdx.x & 48) == 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[threadIdx.x >> 6][l * 4 + e] = v[e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = 0.f;
#pragma unroll
        for (int q = 0; q < kWide / 64; ++q) v[e] += red[q][l * 4 + e];
    }
}

// any number of channels and positions: the tile is read again for each pass
template <typename TX, typename TY>
__global__ __launch_bounds__(kWide) void norm_nchw_fwd_wide_kernel(const NormArgs a, int tiles_p)
{
    __shared__ float red[kWide / 64][kPos];
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes, C = a.C;
    const float fc = float(C);
    for (int64_t t = blockIdx.x; t < a.N * tiles_p; t += gridDim.x) {
        const TilePos at(t, tiles_p, l, a);
        const TX *x = static_cast<const TX *>(a.x) + at.base + at.p;
        TY *y = static_cast<TY *>(a.out) + at.base + at.p;
        float v[4], mean[4] = {}, var[4] = {}, rstd[4];
        for (int c = g; c < C; c += kWideGroups) {
            load_some<4>(x + c * a.P, at.left, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) mean[e] += v[e];
        }
        chan_sum(mean, red);
#pragma unroll
        for (int e = 0; e < 4; ++e) mean[e] /= fc;
        for (int c = g; c < C; c += kWideGroups) {
            load_some<4>(x + c * a.P, at.left, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) var[e] += (v[e] - mean[e]) * (v[e] - mean[e]);
        }
        chan_sum(var, red);
#pragma unroll
        for (int e = 0; e < 4; ++e) rstd[e] = 1.f / sqrtf(var[e] / fc + a.eps);
        if (g == 0 && a.mean) {
            store_some<4>(a.mean + at.n * a.P + at.p, at.left, mean);
            store_some<4>(a.rstd + at.n * a.P + at.p, at.left, rstd);
        }
        for (int c = g; c < C; c += kWideGroups) {
            const float w = a.weight ? a.weight[c] : 1.f, b = a.bias ? a.bias[c] : 0.f;
            load_some<4>(x + c * a.P, at.left, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (v[e] - mean[e]) * rstd[e] * w + b;
            if (a.drop.threshold) drop_run<4>(at.base + c * a.P + at.p, a.drop, v);
            store_some<4>(y + c * a.P, at.left, v);
        }
    }
}

template <typename TX, typename TY>
__global__ __launch_bounds__(kWide) void norm_nchw_bwd_wide_kernel(const NormArgs a, int tiles_p)
{
    __shared__ float red[kWide / 64][kPos];
    const int l = threadIdx.x % kPosLanes, g = threadIdx.x / kPosLanes, C = a.C;
    const float fc = float(C);
    for (int64_t t = blockIdx.x; t < a.N * tiles_p; t += gridDim.x) {
        const TilePos at(t, tiles_p, l, a);
        const TX *x = static_cast<const TX *>(a.x) + at.base + at.p;
        const TY *dy = static_cast<const TY *>(a.dy) + at.base + at.p;
        TX *dx = static_cast<TX *>(a.out) + at.base + at.p;
        float mean[4], rstd[4], h[4], z[4], s1[4] = {}, s2[4] = {};
        load_some<4>(a.mean + at.n * a.P + at.p, at.left, mean);
        load_some<4>(a.rstd + at.n * a.P + at.p, at.left, rstd);
        auto load = [&](int c) {                       // xhat and dz * weight
            const float w = a.weight ? a.weight[c] : 1.f;
            load_some<4>(x + c * a.P, at.left, h);
            load_some<4>(dy + c * a.P, at.left, z);
            if (a.drop.threshold) drop_run<4>(at.base + c * a.P + at.p, a.drop, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[e] = (h[e] - mean[e]) * rstd[e];
                z[e] *= w;
            }
        };
        for (int c = g; c < C; c += kWideGroups) {
            load(c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s1[e] += z[e];
                s2[e] += z[e] * h[e];
            }
        }
        chan_sum(s1, red);
        chan_sum(s2, red);
        for (int c = g; c < C; c += kWideGroups) {
            load(c);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = rstd[e] * (z[e] - s1[e] / fc - h[e] * (s2[e] / fc));
            store_some<4>(dx + c * a.P, at.left, z);
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

// Waves per workgroup and channels per thread: channels in registers, as few as
// hold them all, since fewer registers mean more tiles in flight; kr 0: read
// again for each pass
struct Hold {
    int waves, kr;
};
Hold hold_of(int64_t C, int64_t P)
{
    if (P < 4 || C * P >= int64_t(1) << 30) return {0, 0};
    if (C <= 64) return {4, 4};
    if (C <= 128) return {4, 8};
    if (C <= 256) return {8, 8};
    if (C <= 512) return {8, 16};
    return {0, 0};
}

template <typename F>
hipError_t with_hold(const Hold &h, bool exact, F f)
{
    using std::integral_constant;
    const auto call = [&](auto w, auto k) { return exact ? f(w, k, std::true_type{}) : f(w, k, std::false_type{}); };
    if (h.waves == 4 && h.kr == 4) return call(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    if (h.waves == 4) return call(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    if (h.kr == 8) return call(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    return call(integral_constant<int, 8>{}, integral_constant<int, 16>{});
}

constexpr int64_t kMaxBlocksFwd = 4096, kMaxBlocksBwd = 512, kImageSplits = 16;

int64_t tiles_of(int64_t N, int64_t P) { return N * ((P + kPos - 1) / kPos); }

}  // namespace

int64_t norm_nchw_partials(int64_t N, int64_t C, int64_t P)
{
    if (!hold_of(C, P).kr) return kImageSplits;
    return std::max<int64_t>(1, std::min(tiles_of(N, P), kMaxBlocksBwd));
}

hipError_t launch_norm_nchw_fwd(const NormArgs &a, hipStream_t s)
{
    const Hold h = hold_of(a.C, a.P);
    const int64_t tiles = tiles_of(a.N, a.P);
    const int tiles_p = int((a.P + kPos - 1) / kPos);
    return with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (!h.kr || tiles > INT32_MAX) {
            const dim3 grid(unsigned(std::min(tiles, kMaxBlocksFwd)));
            hipLaunchKernelGGL((norm_nchw_fwd_wide_kernel<TX, TY>), grid, dim3(kWide), 0, s, a, tiles_p);
            return hipGetLastError();
        }
        return with_hold(h, a.P % 4 == 0, [&](auto w, auto k, auto exact) {
            constexpr int WAVES = decltype(w)::value, KR = decltype(k)::value;
            hipLaunchKernelGGL((norm_nchw_fwd_kernel<TX, TY, WAVES, KR, decltype(exact)::value>),
                               dim3(unsigned(tiles)), dim3(WAVES * 64), 0, s, a, tiles_p);
            return hipGetLastError();
        });
    });
}

hipError_t launch_norm_nchw_bwd(const NormArgs &a, hipStream_t s)
{
    const Hold h = hold_of(a.C, a.P);
    const int64_t blocks = norm_nchw_partials(a.N, a.C, a.P);
    const int tiles_p = int((a.P + kPos - 1) / kPos);
    hipError_t e = with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (h.kr)
            return with_hold(h, a.P % 4 == 0, [&](auto w, auto k, auto exact) {
                constexpr int WAVES = decltype(w)::value, KR = decltype(k)::value;
                hipLaunchKernelGGL((norm_nchw_bwd_kernel<TX, TY, WAVES, KR, decltype(exact)::value>),
                                   dim3(unsigned(blocks)), dim3(WAVES * 64), 0, s, a, tiles_p);
                return hipGetLastError();
            });
        const dim3 grid(unsigned(std::max<int64_t>(1, std::min(tiles_of(a.N, a.P), kMaxBlocksFwd))));
        hipLaunchKernelGGL((norm_nchw_bwd_wide_kernel<TX, TY>), grid, dim3(kWide), 0, s, a, tiles_p);
        const hipError_t e1 = hipGetLastError();
        if (e1 != hipSuccess || !a.partial) return e1;
        hipLaunchKernelGGL((norm_planes_kernel<TX, TY>), dim3(unsigned((a.C + 3) / 4), unsigned(blocks)),
                           dim3(256), 0, s, a);
        return hipGetLastError();
    });
    if (e != hipSuccess || !a.partial) return e;
    return launch_norm_reduce(a.partial, blocks, a.C, a.dweight, a.dbias, s);
}

}  // namespace im2win
