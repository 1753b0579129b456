// Layer norm over contiguous channels (NHWC rows): forward, backward and the
// weight-gradient reduction. All bound by HBM: forward reads x and writes y
// once, backward reads x and dy and writes dx once.
//
// A row is held in registers by a group of LPR lanes, KCH chunks of 8
// channels per lane (chunk i of lane l covers channels (i*LPR + l)*8 ..), so
// the mean, the squared deviations around it and the output need one read of
// the row; the channels of a lane are the same for every row, so weight and
// bias, and backward the lane's share of dweight and dbias, stay in registers
// over all the rows a group takes. Each workgroup writes one row of partial
// weight gradients, a second kernel adds those in a fixed order.
// Rows wider than the largest group holds are read again for each pass.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm_common.hpp"

namespace im2win {
namespace {

constexpr int kThreads = 256;

// sum of (a, b) over the LPR lanes of a row. One barrier per call for a
// workgroup-wide row: `slot` alternates between calls, so a wave that is
// ahead writes the other slot.
template <int LPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*red)[2][kThreads / 64], int slot)
{
    a = lane_sum<(LPR < 64 ? LPR : 64)>(a);
    b = lane_sum<(LPR < 64 ? LPR : 64)>(b);
    if constexpr (LPR > 64) {
        if ((threadIdx.x & 63) == 0) {
            red[slot][0][threadIdx.x >> 6] = a;
            red[slot][1][threadIdx.x >> 6] = b;
        }
        __syncthreads();
        a = 0.f;
        b = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) {
            a += red[slot][0][w];
            b += red[slot][1][w];
        }
    }
}

template <typename TX, typename TY, int LPR, int KCH>
__global__ __launch_bounds__(kThreads) void norm_rows_fwd_kernel(const NormArgs a)
{
    constexpr int G = kThreads / LPR;          // rows in flight per workgroup
    __shared__ float red[2][2][kThreads / 64];
    const int l = threadIdx.x % LPR, C = a.C;
    const TX *x = static_cast<const TX *>(a.x);
    TY *y = static_cast<TY *>(a.out);
    const float fc = float(C);

    float w[KCH][8], b[KCH][8];
    int left[KCH];                             // channels of each chunk (<= 0: none)
#pragma unroll
    for (int i = 0; i < KCH; ++i) {
        const int c = (i * LPR + l) * 8;
        left[i] = C - c;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[i][e] = 1.f;
            b[i][e] = 0.f;
        }
        if (a.weight) load_some<8>(a.weight + c, left[i], w[i]);
        if (a.bias) load_some<8>(a.bias + c, left[i], b[i]);
    }

    for (int64_t r = int64_t(blockIdx.x) * G + threadIdx.x / LPR; r < a.N; r += int64_t(gridDim.x) * G) {
        float v[KCH][8], sum = 0.f, sq = 0.f, zero = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            load_some<8>(x + r * a.ldx + (i * LPR + l) * 8, left[i], v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[i][e];
        }
        row_sum2<LPR>(sum, zero, red, 0);
        const float mean = sum / fc;
#pragma unroll
        for (int i = 0; i < KCH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = e < left[i] ? v[i][e] - mean : 0.f;
                sq += v[i][e] * v[i][e];
            }
        row_sum2<LPR>(sq, zero, red, 1);
        const float rstd = 1.f / sqrtf(sq / fc + a.eps);
        if (l == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            if (left[i] <= 0) continue;
            const int c = (i * LPR + l) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * rstd * w[i][e] + b[i][e];
            if (a.drop.threshold) drop_run<8>(r * C + c, a.drop, v[i]);
            store_some<8>(y + r * a.ldo + c, left[i], v[i]);
        }
    }
}

// rows wider than 256 lanes hold: one workgroup per row, three reads of it
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_rows_fwd_wide_kernel(const NormArgs a)
{
    __shared__ float red[2][2][kThreads / 64];
    const int C = a.C;
    const float fc = float(C);
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + r * a.ldx;
        TY *y = static_cast<TY *>(a.out) + r * a.ldo;
        float sum = 0.f, sq = 0.f, zero = 0.f, v[8];
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            load_some<8>(x + c, C - c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[e];
        }
        row_sum2<kThreads>(sum, zero, red, 0);
        const float mean = sum / fc;
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            load_some<8>(x + c, C - c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sq += e < C - c ? (v[e] - mean) * (v[e] - mean) : 0.f;
        }
        row_sum2<kThreads>(sq, zero, red, 1);
        const float rstd = 1.f / sqrtf(sq / fc + a.eps);
        if (threadIdx.x == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            float w[8], b[8];
            load_some<8>(x + c, C - c, v);
            if (a.weight) load_some<8>(a.weight + c, C - c, w);
            if (a.bias) load_some<8>(a.bias + c, C - c, b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = (v[e] - mean) * rstd * (a.weight ? w[e] : 1.f) + (a.bias ? b[e] : 0.f);
            if (a.drop.threshold) drop_run<8>(r * C + c, a.drop, v);
            store_some<8>(y + c, C - c, v);
        }
    }
}

template <typename TX, typename TY, int LPR, int KCH>
__global__ __launch_bounds__(kThreads) void norm_rows_bwd_kernel(const NormArgs a)
{
    constexpr int G = kThreads / LPR;
    __shared__ float red[2][2][kThreads / 64];
    __shared__ float part[G * LPR * KCH * 8];
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR, C = a.C;
    const TX *x = static_cast<const TX *>(a.x);
    const TY *dy = static_cast<const TY *>(a.dy);
    TX *dx = static_cast<TX *>(a.out);
    const float fc = float(C);

    float w[KCH][8], dw[KCH][8], db[KCH][8];
    int left[KCH];
#pragma unroll
    for (int i = 0; i < KCH; ++i) {
        const int c = (i * LPR + l) * 8;
        left[i] = C - c;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[i][e] = 1.f;
            dw[i][e] = 0.f;
            db[i][e] = 0.f;
        }
        if (a.weight) load_some<8>(a.weight + c, left[i], w[i]);
    }

    int slot = 0;
    for (int64_t r = int64_t(blockIdx.x) * G + g; r < a.N; r += int64_t(gridDim.x) * G) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float h[KCH][8], z[KCH][8], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8;
            load_some<8>(x + r * a.ldx + c, left[i], h[i]);
            load_some<8>(dy + r * a.ldy + c, left[i], z[i]);
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            if (a.drop.threshold && left[i] > 0) drop_run<8>(r * C + (i * LPR + l) * 8, a.drop, z[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = e < left[i] ? (h[i][e] - mean) * rstd : 0.f;
                dw[i][e] += z[i][e] * h[i][e];
                db[i][e] += z[i][e];
                z[i][e] *= w[i][e];
                s1 += z[i][e];
                s2 += z[i][e] * h[i][e];
            }
        }
        row_sum2<LPR>(s1, s2, red, slot);
        slot ^= 1;
        s1 /= fc;
        s2 /= fc;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            if (left[i] <= 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = rstd * (z[i][e] - s1 - h[i][e] * s2);
            store_some<8>(dx + r * a.ldo + (i * LPR + l) * 8, left[i], z[i]);
        }
    }

    if (!a.partial) return;
    // the workgroup's groups added in order, dweight first, then dbias
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KCH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) part[(g * KCH + i) * LPR * 8 + l * 8 + e] = k ? db[i][e] : dw[i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += kThreads) {
            float t = 0.f;
            for (int q = 0; q < G; ++q) t += part[q * KCH * LPR * 8 + c];
            a.partial[(int64_t(blockIdx.x) * 2 + k) * C + c] = t;
        }
    }
}

template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_rows_bwd_wide_kernel(const NormArgs a)
{
    __shared__ float red[2][2][kThreads / 64];
    const int C = a.C;
    const float fc = float(C);
    int slot = 0;
    for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x) {
        const TX *x = static_cast<const TX *>(a.x) + r * a.ldx;
        const TY *dy = static_cast<const TY *>(a.dy) + r * a.ldy;
        TX *dx = static_cast<TX *>(a.out) + r * a.ldo;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float h[8], z[8], w[8], s1 = 0.f, s2 = 0.f;
        auto load = [&](int c) {
            load_some<8>(x + c, C - c, h);
            load_some<8>(dy + c, C - c, z);
            if (a.weight) load_some<8>(a.weight + c, C - c, w);
            if (a.drop.threshold) drop_run<8>(r * C + c, a.drop, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = e < C - c ? (h[e] - mean) * rstd : 0.f;
                if (a.weight) z[e] *= w[e];
            }
        };
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            load(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s1 += z[e];
                s2 += z[e] * h[e];
            }
        }
        row_sum2<kThreads>(s1, s2, red, slot);
        slot ^= 1;
        s1 /= fc;
        s2 /= fc;
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            load(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = rstd * (z[e] - s1 - h[e] * s2);
            store_some<8>(dx + c, C - c, z);
        }
    }
}

// the wide rows' weight gradients: a workgroup takes 512 channels and every
// gridDim.y-th group of four rows, a wave one row at a time
template <typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void norm_cols_kernel(const NormArgs a)
{
    __shared__ float part[4][512];
    const int C = a.C, wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int c0 = blockIdx.x * 512, c = c0 + l * 8;
    float dw[8] = {}, db[8] = {};
    if (c < C) {
        for (int64_t r = int64_t(blockIdx.y) * 4 + wave; r < a.N; r += int64_t(gridDim.y) * 4) {
            float h[8], z[8];
            load_some<8>(static_cast<const TX *>(a.x) + r * a.ldx + c, C - c, h);
            load_some<8>(static_cast<const TY *>(a.dy) + r * a.ldy + c, C - c, z);
            if (a.drop.threshold) drop_run<8>(r * C + c, a.drop, z);
            const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[e] += z[e] * (h[e] - mean) * rstd;
                db[e] += z[e];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) part[wave][l * 8 + e] = k ? db[e] : dw[e];
        __syncthreads();
        for (int i = threadIdx.x; i < 512 && c0 + i < C; i += kThreads)
            a.partial[(int64_t(blockIdx.y) * 2 + k) * C + c0 + i] =
                (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
    }
}

// dweight, dbias: 16 columns of [rows][2*C] per workgroup, 64 row groups
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float *partial, int rows, int C,
                                                           float *dweight, float *dbias)
{
    __shared__ float part[64][17];
    const int col = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int64_t k = int64_t(blockIdx.x) * 16 + col;
    float t = 0.f;
    if (k < 2 * int64_t(C))
#pragma unroll 4
        for (int r = g; r < rows; r += 64) t += partial[int64_t(r) * 2 * C + k];
    part[g][col] = t;
    __syncthreads();
    for (int m = 32; m > 0; m >>= 1) {
        if (g < m) part[g][col] += part[g + m][col];
        __syncthreads();
    }
    if (g == 0 && k < 2 * int64_t(C)) (k < C ? dweight : dbias)[k < C ? k : k - C] = part[0][col];
}

// The group that holds a row of C channels: as few lanes per row as keep it to
// one chunk each (so narrow rows fill whole waves), past one wave's width up
// to four chunks per lane, then the whole workgroup. wide: no group holds it.
struct Group {
    int lpr, kch;
};
Group group_of(int64_t C)
{
    const int64_t ch = (C + 7) / 8;
    if (ch <= 8) return {8, 1};
    if (ch <= 16) return {16, 1};
    if (ch <= 32) return {32, 1};
    if (ch <= 64) return {64, 1};
    if (ch <= 128) return {64, 2};
    if (ch <= 256) return {256, 1};
    if (ch <= 512) return {256, 2};
    if (ch <= 1024) return {256, 4};
    return {0, 0};
}

template <typename F>
hipError_t with_group(const Group &g, F f)
{
    using std::integral_constant;
    if (g.lpr == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (g.lpr == 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (g.lpr == 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (g.lpr == 64 && g.kch == 1) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (g.lpr == 64) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (g.kch == 1) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (g.kch == 2) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
}

constexpr int64_t kMaxBlocksFwd = 2048;
constexpr int64_t kMaxBlocksBwd = 512;
constexpr int64_t kColSplits = 32;

}  // namespace

int64_t norm_rows_partials(int64_t N, int64_t C)
{
    const Group g = group_of(C);
    if (!g.lpr) return kColSplits;
    const int64_t per = kThreads / g.lpr;
    return std::max<int64_t>(1, std::min((N + per - 1) / per, kMaxBlocksBwd));
}

hipError_t launch_norm_rows_fwd(const NormArgs &a, hipStream_t s)
{
    const Group g = group_of(a.C);
    return with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (!g.lpr) {
            const dim3 grid(unsigned(std::min(a.N, kMaxBlocksFwd)));
            hipLaunchKernelGGL((norm_rows_fwd_wide_kernel<TX, TY>), grid, dim3(kThreads), 0, s, a);
            return hipGetLastError();
        }
        return with_group(g, [&](auto lpr, auto kch) {
            constexpr int LPR = decltype(lpr)::value, KCH = decltype(kch)::value;
            const int64_t per = kThreads / LPR;
            const dim3 grid(unsigned(std::min((a.N + per - 1) / per, kMaxBlocksFwd)));
            hipLaunchKernelGGL((norm_rows_fwd_kernel<TX, TY, LPR, KCH>), grid, dim3(kThreads), 0, s, a);
            return hipGetLastError();
        });
    });
}

hipError_t launch_norm_rows_bwd(const NormArgs &a, hipStream_t s)
{
    const Group g = group_of(a.C);
    const int64_t blocks = norm_rows_partials(a.N, a.C);
    hipError_t e = with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (!g.lpr) {
            const dim3 grid(unsigned(std::max<int64_t>(1, std::min(a.N, kMaxBlocksFwd))));
            hipLaunchKernelGGL((norm_rows_bwd_wide_kernel<TX, TY>), grid, dim3(kThreads), 0, s, a);
            hipError_t e1 = hipGetLastError();
            if (e1 != hipSuccess || !a.partial) return e1;
            hipLaunchKernelGGL((norm_cols_kernel<TX, TY>), dim3(unsigned((a.C + 511) / 512), unsigned(blocks)),
                               dim3(kThreads), 0, s, a);
            return hipGetLastError();
        }
        return with_group(g, [&](auto lpr, auto kch) {
            constexpr int LPR = decltype(lpr)::value, KCH = decltype(kch)::value;
            hipLaunchKernelGGL((norm_rows_bwd_kernel<TX, TY, LPR, KCH>), dim3(unsigned(blocks)),
                               dim3(kThreads), 0, s, a);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || !a.partial) return e;
    return launch_norm_reduce(a.partial, blocks, a.C, a.dweight, a.dbias, s);
}

hipError_t launch_norm_reduce(const float *partial, int64_t rows, int C, float *dweight, float *dbias,
                              hipStream_t s)
{
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(unsigned((2 * int64_t(C) + 15) / 16)), dim3(1024), 0, s,
                       partial, int(rows), C, dweight, dbias);
    return hipGetLastError();
}

}  // namespace im2win
