// Layer norm over the channels of NCHW feature maps: forward and backward.
// Bound by HBM like the row kernels; here a position's channels are P elements
// apart, so a workgroup takes a tile of consecutive positions of one image and
// all its channels. Thread (g, l) holds PV positions from PV l on (one vector load
// per channel, PL lanes reading consecutive memory) of KR channels g, g + groups,
// ...; a wave adds its channels in registers, the waves' sums meet in LDS.
// Backward, a thread's share of dweight and dbias stays in registers over all
// tiles the workgroup takes. Maps of more than 1024 channels, or fewer than 4
// positions, are read again for each pass. Forward 64 channels of 56 x 56, 32
// images, fp32 to fp16 11.5 us (3.4 TB/s: one wave of tiles); backward 256 channels
// of 56 x 56, 64 images, fp32 124 us (5.0 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm_common.hpp"

namespace im2win {
namespace {

constexpr int kPosLanes = 16, kPos = 64;       // lanes, and positions of a tile of 4 per lane

// v[e] over the lanes of a wave that hold the same positions, every PL-th
template <int PV, int PL = kPosLanes>
__device__ __forceinline__ void wave_chan_sum(float (&v)[PV])
{
#pragma unroll
    for (int e = 0; e < PV; ++e) {
        const uint32_t u = __float_as_uint(v[e]);
        const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        const uint32_t w = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
        const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
        v[e] = __uint_as_float(q[0]) + __uint_as_float(q[1]);
        if constexpr (PL == 8)                     // lane i and i + 8 of 16: a rotation by 8
            v[e] += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v[e]), 0x128, 0xf, 0xf, true));
    }
}

// where this thread's positions lie, PV of them per lane, PL lanes a channel
template <int PV, int PL = kPosLanes>
struct TilePos {
    int64_t n, p, base;      // image, first position, offset of channel 0 there
    int left;                // positions that exist (<= 0: none)
    __device__ __forceinline__ TilePos(int64_t t, int tiles_p, int l, const NormArgs &a)
    {
        n = t / tiles_p;
        p = (t - n * tiles_p) * (PL * PV) + l * PV;
        left = int(min(int64_t(PV), a.P - p));
        base = n * a.C * a.P;
    }
};

template <bool EXACT, int PV, typename T>
__device__ __forceinline__ void store_pos(T *p, int left, const float (&f)[PV])
{
    if constexpr (EXACT) {
        if (left > 0) store_vec<PV>(p, f);
    } else {
        store_some<PV>(p, left, f);
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

// where positions p .. p + PV - 1 of a channel are read from, and how far that is
// before p (see load_row)
template <int PV>
struct Window {
    uint32_t at;
    int shift;
    __device__ __forceinline__ Window(int64_t p, int64_t P)
    {
        const int64_t q = p < P - PV ? p : P - PV;
        at = uint32_t(q);
        shift = int(p - q < PV ? p - q : PV);
    }
};

// Dropout of a tile: the blocks of 16 * PV positions of KR channels overlap from
// lane to lane, so the lanes of a channel group make each block once and pass
// the kept bits through LDS (a Philox block per lane and channel, or two where P
// is no multiple of 4, is what these kernels waited for: 384 channels of 7 x 7,
// 2354 images, f16 backward 264 us, so 176; with P a multiple of 4 it is even,
// 164 channels of 56 x 56, 97 images forward 93 and 101).
template <int KR, int PV, int PL = kPosLanes>
struct TileDrop {
    static constexpr int BLOCKS = PL * PV / 8 + 1;                    // that a channel's positions may touch
    static constexpr int ROUNDS = (KR * BLOCKS + PL - 1) / PL;
    static constexpr int KW = 32 / PV, WORDS = (KR + KW - 1) / KW;    // channels per word of kept bits
    static constexpr int BYTES = ROUNDS * PL + 4;                     // of a group
    uint32_t keep[WORDS];

    // the kept bits of channels g, g + G, ..; e0: the tile's first element in channel 0
    __device__ __forceinline__ void make(uint8_t *bytes, int64_t e0, uint32_t P, int G, const DropSpec &d)
    {
        const int l = threadIdx.x % PL, g = threadIdx.x / PL;
        uint8_t *mine = bytes + g * BYTES;
        __builtin_amdgcn_sched_barrier(0);         // between the loads and their first use
        before();
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int job = r * PL + l, i = job / BLOCKS;
            const uint64_t e = uint64_t(e0 + uint32_t(g + i * G) * int64_t(P));
            mine[job] = uint8_t(keep_bits((e >> 3) + (job - i * BLOCKS), d));
        }
        before();
#pragma unroll
        for (int k = 0; k < WORDS; ++k) keep[k] = 0;
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const uint32_t o = (uint32_t(e0 + uint32_t(g + i * G) * int64_t(P)) & 7) + l * PV;
            const uint8_t *b = mine + i * BLOCKS + (o >> 3);
            keep[i / KW] |= ((b[0] | b[1] << 8) >> (o & 7) & ((1u << PV) - 1)) << (i % KW * PV);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ bool kept(int i, int e) const { return (keep[i / KW] >> (i % KW * PV + e)) & 1; }

private:
    // a group lies within a wave, whose LDS accesses are in order
    static __device__ __forceinline__ void before()
    {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
};

// One tile, first + blockIdx.x. WAVES waves, 64 / PL * WAVES channel groups; EXACT: P is
// a multiple of PV
template <typename TX, typename TY, int WAVES, int KR, int PV, int PL, bool EXACT>
__global__ __launch_bounds__(WAVES * 64) void norm_nchw_fwd_kernel(const NormArgs a, int tiles_p, int64_t first)
{
    constexpr int GW = 64 / PL, G = WAVES * GW;
    __shared__ __align__(16) float red[2][WAVES][PL * PV];    // mean, squares
    const int l = threadIdx.x % PL, g = threadIdx.x / PL, wave = threadIdx.x >> 6, C = a.C;
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
        for (int i = 0; i < KR; ++i) n += max(0, min(GW, C - i * G - q * GW));
        return float(n);
    };
    const TilePos<PV, PL> at(first + blockIdx.x, tiles_p, l, a);
    const TX *x = static_cast<const TX *>(a.x) + at.base;
    TY *y = static_cast<TY *>(a.out) + at.base;
    const Window<PV> win(at.p, a.P);
    TileDrop<KR, PV, PL> drop;
    __shared__ uint8_t bytes[G * TileDrop<KR, PV, PL>::BYTES];
    // channels past the last read that one and count nowhere
    Raw<TX, PV> q[KR];
#pragma unroll
    for (int i = 0; i < KR; ++i)
        q[i] = load_raw<TX, PV>(at_offset(x, uint32_t(min(g + i * G, C - 1)) * P + win.at));
    if (a.drop.threshold) drop.make(bytes, at.base + at.p - l * PV, P, G, a.drop);
    if constexpr (!EXACT)
#pragma unroll
        for (int i = 0; i < KR; ++i) shift_down(q[i], win.shift);
    float v[KR][PV], mean[PV] = {}, sq[PV] = {};
#pragma unroll
    for (int i = 0; i < KR; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            v[i][e] = element(q[i], e);
            mean[e] += g + i * G < C ? v[i][e] : 0.f;
        }
    // a wave's own mean and squared deviations, joined with one barrier:
    // sum (x - mean)^2 = sum_w [Q_w + n_w (mean_w - mean)^2]
    wave_chan_sum<PV, PL>(mean);
    const float nw = fmaxf(count(wave), 1.f);
#pragma unroll
    for (int e = 0; e < PV; ++e) mean[e] /= nw;
#pragma unroll
    for (int i = 0; i < KR; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            const float d = v[i][e] - mean[e];
            sq[e] += g + i * G < C ? d * d : 0.f;
        }
    wave_chan_sum<PV, PL>(sq);
    if ((threadIdx.x & 63) < PL)
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            red[0][wave][l * PV + e] = mean[e];
            red[1][wave][l * PV + e] = sq[e];
        }
    __syncthreads();
    float rstd[PV], m[PV] = {}, s[PV] = {};
#pragma unroll 4
    for (int k = 0; k < WAVES; ++k) {
        const float n = count(k);
#pragma unroll
        for (int e = 0; e < PV; ++e) m[e] += red[0][k][l * PV + e] * n;
    }
#pragma unroll
    for (int e = 0; e < PV; ++e) m[e] /= fc;
#pragma unroll 4
    for (int k = 0; k < WAVES; ++k) {
        const float n = count(k);
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            const float d = red[0][k][l * PV + e] - m[e];
            s[e] += red[1][k][l * PV + e] + n * d * d;
        }
    }
#pragma unroll
    for (int e = 0; e < PV; ++e) {
        mean[e] = m[e];
        rstd[e] = 1.f / sqrtf(s[e] / fc + a.eps);
    }
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        const int c = g + i * G;
#pragma unroll
        for (int e = 0; e < PV; ++e) v[i][e] = (v[i][e] - mean[e]) * rstd[e] * w[i] + b[i];
        if (a.drop.threshold)
#pragma unroll
            for (int e = 0; e < PV; ++e) v[i][e] = drop.kept(i, e) ? v[i][e] * a.drop.scale : 0.f;
        store_pos<EXACT>(at_offset(y, c * P + uint32_t(at.p)), c < C ? at.left : 0, v[i]);
    }
    if (g == 0 && a.mean) {
        store_some<PV>(a.mean + at.n * a.P + at.p, at.left, mean);
        store_some<PV>(a.rstd + at.n * a.P + at.p, at.left, rstd);
    }
}

template <typename TX, typename TY, int WAVES, int KR, int PV, int PL, bool EXACT, bool DROP>
__global__ __launch_bounds__(WAVES * 64) void norm_nchw_bwd_kernel(const NormArgs a, int tiles_p)
{
    constexpr int G = WAVES * 64 / PL;
    __shared__ __align__(16) float red[2][2][WAVES][PL * PV];
    const int l = threadIdx.x % PL, g = threadIdx.x / PL, wave = threadIdx.x >> 6, C = a.C;
    const float fc = float(C);
    const int64_t tiles = a.N * tiles_p;
    float w[KR], dw[KR], db[KR];
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        w[i] = a.weight ? a.weight[min(g + i * G, C - 1)] : 1.f;
        dw[i] = db[i] = 0.f;
    }
    int slot = 0;
    TileDrop<KR, PV, PL> drop;
    __shared__ uint8_t bytes[DROP ? G * TileDrop<KR, PV, PL>::BYTES : 1];
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const TilePos<PV, PL> at(t, tiles_p, l, a);
        // opaque, so that no offset of a channel is kept in registers over the tiles
        uint32_t P = uint32_t(a.P);
        asm volatile("" : "+s"(P));
        const TX *x = static_cast<const TX *>(a.x) + at.base;
        const TY *dy = static_cast<const TY *>(a.dy) + at.base;
        TX *dx = static_cast<TX *>(a.out) + at.base;
        const Window<PV> win(at.p, a.P);
        Raw<float, PV> rm = load_row<float, PV, EXACT>(a.mean + at.n * a.P, at.p, a.P);
        Raw<float, PV> rr = load_row<float, PV, EXACT>(a.rstd + at.n * a.P, at.p, a.P);
        Raw<TX, PV> qx[KR];
        Raw<TY, PV> qy[KR];
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const uint32_t o = uint32_t(min(g + i * G, C - 1)) * P + win.at;
            qx[i] = load_raw<TX, PV>(at_offset(x, o));
            qy[i] = load_raw<TY, PV>(at_offset(dy, o));
        }
        if constexpr (DROP) drop.make(bytes, at.base + at.p - l * PV, P, G, a.drop);
        if constexpr (!EXACT)
#pragma unroll
            for (int i = 0; i < KR; ++i) {
                shift_down(qx[i], win.shift);
                shift_down(qy[i], win.shift);
            }
        // a position past the end has mean, rstd and dy 0, a channel past the last
        // dy 0: they add nothing (not EXACT: the shift has cleared the positions)
        const uint32_t pos = !EXACT || at.left > 0 ? ~0u : 0u;
        keep_if(rm, pos);
        keep_if(rr, pos);
#pragma unroll
        for (int i = 0; i < KR; ++i) keep_if(qy[i], g + i * G < C ? pos : 0u);
        // xhat and dz of channel i: formed from the raw values in both passes, which
        // takes half the registers of keeping them; a dropout mask is kept (a bit)
        auto form = [&](int i, float (&h)[PV], float (&z)[PV]) {
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                h[e] = (element(qx[i], e) - element(rm, e)) * element(rr, e);
                z[e] = element(qy[i], e);
                if constexpr (DROP) z[e] = drop.kept(i, e) ? z[e] * a.drop.scale : 0.f;
            }
        };
        float s1[PV] = {}, s2[PV] = {};
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            float h[PV], z[PV];
            form(i, h, z);
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                dw[i] += z[e] * h[e];
                db[i] += z[e];
                s1[e] += z[e] * w[i];
                s2[e] += z[e] * w[i] * h[e];
            }
            __builtin_amdgcn_sched_barrier(0);     // one channel's values at a time
        }
        wave_chan_sum<PV, PL>(s1);
        wave_chan_sum<PV, PL>(s2);
        if ((threadIdx.x & 63) < PL)
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                red[slot][0][wave][l * PV + e] = s1[e];
                red[slot][1][wave][l * PV + e] = s2[e];
            }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < PV; ++e) s1[e] = s2[e] = 0.f;
#pragma unroll 4
        for (int k = 0; k < WAVES; ++k)
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                s1[e] += red[slot][0][k][l * PV + e];
                s2[e] += red[slot][1][k][l * PV + e];
            }
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            s1[e] /= fc;
            s2[e] /= fc;
        }
        slot ^= 1;
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const int c = g + i * G;
            float o[PV], h[PV], z[PV];
            arrive(qx[i]);                     // opaque: formed anew, not kept since the first pass
            arrive(qy[i]);
            form(i, h, z);
#pragma unroll
            for (int e = 0; e < PV; ++e) o[e] = element(rr, e) * (z[e] * w[i] - s1[e] - h[e] * s2[e]);
            store_pos<EXACT>(at_offset(dx, c * P + uint32_t(at.p)), c < C ? at.left : 0, o);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < KR; ++i) {
        const float u = lane_sum<PL>(dw[i]), v = lane_sum<PL>(db[i]);
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

// positions p .. p + 3 of a channel's row of P, zeros past its end
template <typename T>
__device__ __forceinline__ void load_pos(const T *row, int64_t p, int64_t P, float (&f)[4])
{
    if (P >= 4) {                              // wave-uniform
        const Raw<T, 4> r = load_row<T, 4, false>(row, p, P);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = element(r, e);
    } else {
        load_some<4>(row + p, P - p, f);
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
        const TilePos<4> at(t, tiles_p, l, a);
        const TX *x = static_cast<const TX *>(a.x) + at.base;
        TY *y = static_cast<TY *>(a.out) + at.base + at.p;
        float v[4], mean[4] = {}, var[4] = {}, rstd[4];
#pragma unroll 4
        for (int c = g; c < C; c += kWideGroups) {
            load_pos(x + c * a.P, at.p, a.P, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) mean[e] += v[e];
        }
        chan_sum(mean, red);
#pragma unroll
        for (int e = 0; e < 4; ++e) mean[e] /= fc;
#pragma unroll 4
        for (int c = g; c < C; c += kWideGroups) {
            load_pos(x + c * a.P, at.p, a.P, v);
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
#pragma unroll 4
        for (int c = g; c < C; c += kWideGroups) {
            const float w = a.weight ? a.weight[c] : 1.f, b = a.bias ? a.bias[c] : 0.f;
            load_pos(x + c * a.P, at.p, a.P, v);
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
        const TilePos<4> at(t, tiles_p, l, a);
        const TX *x = static_cast<const TX *>(a.x) + at.base;
        const TY *dy = static_cast<const TY *>(a.dy) + at.base;
        TX *dx = static_cast<TX *>(a.out) + at.base + at.p;
        float mean[4], rstd[4], h[4], z[4], s1[4] = {}, s2[4] = {};
        load_some<4>(a.mean + at.n * a.P + at.p, at.left, mean);
        load_some<4>(a.rstd + at.n * a.P + at.p, at.left, rstd);
        auto load = [&](int c) {                       // xhat and dz * weight
            const float w = a.weight ? a.weight[c] : 1.f;
            load_pos(x + c * a.P, at.p, a.P, h);
            load_pos(dy + c * a.P, at.p, a.P, z);
            if (a.drop.threshold) drop_run<4>(at.base + c * a.P + at.p, a.drop, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[e] = (h[e] - mean[e]) * rstd[e];
                z[e] *= w;
            }
        };
#pragma unroll 4
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
#pragma unroll 4
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
    const int l = threadIdx.x & 63, C = a.C;
    for (int c = blockIdx.x * 4 + (threadIdx.x >> 6); c < C; c += gridDim.x * 4) {
        float dw = 0.f, db = 0.f;
        for (int64_t n = blockIdx.y; n < a.N; n += gridDim.y) {
            const int64_t base = (n * C + c) * a.P;
            for (int64_t p = l * 4; p < a.P; p += 256) {
                float h[4], z[4], mean[4], rstd[4];
                load_pos(static_cast<const TX *>(a.x) + base, p, a.P, h);
                load_pos(static_cast<const TY *>(a.dy) + base, p, a.P, z);
                load_pos(a.mean + n * a.P, p, a.P, mean);
                load_pos(a.rstd + n * a.P, p, a.P, rstd);
                if (a.drop.threshold) drop_run<4>(base + p, a.drop, z);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dw += z[e] * (h[e] - mean[e]) * rstd[e];   // 0 past the end
                    db += z[e];
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
}

// Waves per workgroup, channels per thread, positions per lane and lanes per
// channel: channels in registers, as few as hold them all, since fewer registers
// mean more tiles in flight; kr 0: read again for each pass. Past 256 channels
// half the positions (16 channels of 4 positions do not fit the registers
// backward: 384 channels of 56 x 56, bf16, 50 images took 246 us, so 114). Past 512
// half the lanes (744 channels of 56 x 56, 5 images, bf16: backward 71 us when read
// again, 44 so, 16 waves spill; forward 33, 27, 32).
struct Hold {
    int waves, kr, pv, pl;
};
Hold hold_of(int64_t C, int64_t P)
{
    if (P < 4 || C > 1024 || C * P >= int64_t(1) << 30) return {0, 0, 4, 16};
    if (C <= 64) return {4, 4, 4, 16};
    if (C <= 128) return {4, 8, 4, 16};
    if (C <= 256) return {8, 8, 4, 16};
    if (C <= 512) return {8, 16, 2, 16};
    return {8, 16, 2, 8};
}

template <int N>
using Int = std::integral_constant<int, N>;

// f(waves, channels, positions, lanes, exact)
template <typename F>
hipError_t with_hold(const Hold &h, int64_t P, F f)
{
    const auto call = [&](auto w, auto k, auto v, auto l) {
        return P % decltype(v)::value == 0 ? f(w, k, v, l, std::true_type{}) : f(w, k, v, l, std::false_type{});
    };
    if (h.waves == 4 && h.kr == 4) return call(Int<4>{}, Int<4>{}, Int<4>{}, Int<16>{});
    if (h.waves == 4) return call(Int<4>{}, Int<8>{}, Int<4>{}, Int<16>{});
    if (h.kr == 8) return call(Int<8>{}, Int<8>{}, Int<4>{}, Int<16>{});
    if (h.pl == 16) return call(Int<8>{}, Int<16>{}, Int<2>{}, Int<16>{});
    return call(Int<8>{}, Int<16>{}, Int<2>{}, Int<8>{});
}

// Workgroups of the re-reading kernels (1024 to 8192 measure the same: 32 images of 1100
// channels, 28 x 28, bf16, forward 58.6 us) and of the backward one that holds its
// tile, each with a row of partial sums (256 channels of 56 x 56, 64 images, fp32: 121.8,
// 124.3 and 126.9 us with 256, 512 and 1024; 64 channels, 32 images, fp16: 19.4, 15.3 and
// 14.9); parts of the images for the re-reading dweight and dbias (1100 channels of 28 x 28,
// 32 images, bf16: 184, 177 and 177 us with 8, 16 and 32; 2000 images of 7 x 7, fp16: 1513, 1383
// and 1344).
constexpr int64_t kMaxBlocksFwd = 4096, kMaxBlocksBwd = 512, kImageSplits = 16;

int64_t tiles_of_image(int64_t P, const Hold &h) { return (P + h.pl * h.pv - 1) / (h.pl * h.pv); }

}  // namespace

int64_t norm_nchw_partials(int64_t N, int64_t C, int64_t P)
{
    const Hold h = hold_of(C, P);
    if (!h.kr) return kImageSplits;
    return std::max<int64_t>(1, std::min(N * tiles_of_image(P, h), kMaxBlocksBwd));
}

hipError_t launch_norm_nchw_fwd(const NormArgs &a, hipStream_t s)
{
    const Hold h = hold_of(a.C, a.P);
    const int64_t tiles_p = tiles_of_image(a.P, h), tiles = a.N * tiles_p;
    return with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (!h.kr) {
            const dim3 grid(unsigned(std::min(tiles, kMaxBlocksFwd)));
            hipLaunchKernelGGL((norm_nchw_fwd_wide_kernel<TX, TY>), grid, dim3(kWide), 0, s, a, int(tiles_p));
            return hipGetLastError();
        }
        return with_hold(h, a.P, [&](auto w, auto k, auto v, auto l, auto exact) {
            constexpr int WAVES = decltype(w)::value, KR = decltype(k)::value, PV = decltype(v)::value;
            constexpr int PL = decltype(l)::value;
            constexpr int64_t most = max_groups(WAVES * 64);
            for (int64_t first = 0; first < tiles; first += most)
                hipLaunchKernelGGL((norm_nchw_fwd_kernel<TX, TY, WAVES, KR, PV, PL, decltype(exact)::value>),
                                   dim3(unsigned(std::min(tiles - first, most))), dim3(WAVES * 64), 0, s, a,
                                   int(tiles_p), first);
            return hipGetLastError();
        });
    });
}

hipError_t launch_norm_nchw_bwd(const NormArgs &a, hipStream_t s)
{
    const Hold h = hold_of(a.C, a.P);
    const int64_t blocks = norm_nchw_partials(a.N, a.C, a.P);
    const int tiles_p = int(tiles_of_image(a.P, h));
    hipError_t e = with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (h.kr)
            return with_hold(h, a.P, [&](auto w, auto k, auto v, auto l, auto exact) {
                constexpr int WAVES = decltype(w)::value, KR = decltype(k)::value, PV = decltype(v)::value;
                constexpr int PL = decltype(l)::value;
                constexpr bool EXACT = decltype(exact)::value;
                const dim3 grid{unsigned(blocks)};
                if (a.drop.threshold)
                    hipLaunchKernelGGL((norm_nchw_bwd_kernel<TX, TY, WAVES, KR, PV, PL, EXACT, true>), grid,
                                       dim3(WAVES * 64), 0, s, a, tiles_p);
                else
                    hipLaunchKernelGGL((norm_nchw_bwd_kernel<TX, TY, WAVES, KR, PV, PL, EXACT, false>), grid,
                                       dim3(WAVES * 64), 0, s, a, tiles_p);
                return hipGetLastError();
            });
        const dim3 grid(unsigned(std::max<int64_t>(1, std::min(a.N * tiles_p, kMaxBlocksFwd))));
        hipLaunchKernelGGL((norm_nchw_bwd_wide_kernel<TX, TY>), grid, dim3(kWide), 0, s, a, tiles_p);
        const hipError_t e1 = hipGetLastError();
        if (e1 != hipSuccess || !a.partial) return e1;
        const int64_t groups = std::min<int64_t>((int64_t(a.C) + 3) / 4, max_groups(256));
        hipLaunchKernelGGL((norm_planes_kernel<TX, TY>), dim3(unsigned(groups), unsigned(blocks)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
    if (e != hipSuccess || !a.partial) return e;
    return launch_norm_reduce(a.partial, blocks, a.C, a.dweight, a.dbias, s);
}

}  // namespace im2win
