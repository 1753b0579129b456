// Layer norm over contiguous channels (NHWC rows): forward, backward and the
// weight-gradient reduction. All bound by HBM: forward reads x and writes y
// once, backward reads x and dy and writes dx once.
//
// A row is held in registers by a group of LPR lanes, KCH chunks of 8
// channels per lane (chunk i of lane l covers channels (i*LPR + l)*8 ..), so
// the mean, the squared deviations around it and the output need one read of
// the row; the channels of a lane are the same for every row, so weight and
// bias, and backward the lane's share of dweight and dbias, stay in registers
// over all the rows a group takes. The next row's loads are issued before the
// current row is worked on. Each workgroup writes one row of partial
// weight gradients, a second kernel adds those in a fixed order.
// Rows wider than the largest group holds are read again for each pass.
// 32768 rows of 4096 bf16 with dropout: forward 117 us (4.6 TB/s), backward 165 us
// (4.9 TB/s), of which the reduction is 7; 50001 rows of 1001 fp16, whose rows start
// at any even address, backward 67 us (4.5 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm_common.hpp"

namespace im2win {
namespace {

constexpr int kThreads = 256;

// threads of a workgroup whose rows take LPR lanes each
constexpr int threads_of(int lpr) { return lpr > 64 ? lpr : kThreads; }

// sum of (a, b) over the LPR lanes of a row. One barrier per call for a
// workgroup-wide row: `slot` alternates between calls, so a wave that is
// ahead writes the other slot.
template <int LPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*red)[2][threads_of(LPR) / 64], int slot)
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
        for (int w = 0; w < threads_of(LPR) / 64; ++w) {
            a += red[slot][0][w];
            b += red[slot][1][w];
        }
    }
}

// dropout of a chunk, and its store (left: channels from its first one to the
// row's end); EXACT: rows of whole chunks
template <bool EXACT>
__device__ __forceinline__ void drop_chunk(int64_t first, const DropSpec &d, float (&f)[8])
{
    if constexpr (EXACT)
        drop_block(uint64_t(first) >> 3, d, f);
    else
        drop_run<8>(first, d, f);
}
template <bool EXACT, typename T>
__device__ __forceinline__ void store_row(T *p, int left, const Raw<T, 8> &r)
{
    if constexpr (EXACT) {
        if (left > 0) store_raw(p, r);
    } else {
        store_some_raw(p, left, r);
    }
}

// weight and bias (1 and 0 where absent) of channels c .. c + 7: in registers
// for one chunk per lane, else in LDS ([LPR * KCH * 8] floats each)
template <int KCH>
struct Params {
    float own[KCH == 1 ? 8 : 1];
    const float *lds;        // chunk i, half h (4 channels) and lane l at ((2i + h) * LPR + l) * 4: a wave's
                             // 16-byte reads are consecutive

    template <int LPR>
    __device__ __forceinline__ void init(const float *p, float absent, int C, float *buf, int l)
    {
        if constexpr (KCH == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) own[e] = absent;
            if (p) load_some<8>(p + l * 8, C - l * 8, own);
        } else {
            for (int c = threadIdx.x; c < LPR * KCH * 8; c += threads_of(LPR))
                buf[((c / (LPR * 8) * 2 + c / 4 % 2) * LPR + c / 8 % LPR) * 4 + c % 4] = p && c < C ? p[c] : absent;
            lds = buf + l * 4;
        }
    }
    template <int LPR>
    __device__ __forceinline__ void get(int i, float (&f)[8]) const
    {
        if constexpr (KCH == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = own[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = lds[(2 * i + e / 4) * LPR * 4 + e % 4];
        }
    }
};

template <typename TX, typename TY, int LPR, int KCH, bool EXACT>
__global__ __launch_bounds__(threads_of(LPR)) void norm_rows_fwd_kernel(const NormArgs a)
{
    constexpr int G = threads_of(LPR) / LPR;   // rows in flight per workgroup
    constexpr int WAVES = LPR > 64 ? LPR / 64 : 1;     // of a row
    __shared__ float2 red[2][WAVES];
    __shared__ __align__(16) float pw[KCH > 1 ? LPR * KCH * 8 : 1], pb[KCH > 1 ? LPR * KCH * 8 : 1];
    const int l = threadIdx.x % LPR, C = a.C;
    const TX *x = static_cast<const TX *>(a.x);
    TY *y = static_cast<TY *>(a.out);
    const float fc = float(C);
    const int64_t step = int64_t(gridDim.x) * G;
    int64_t r = int64_t(blockIdx.x) * G + threadIdx.x / LPR;

    Raw<TX, 8> q[KCH];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < KCH; ++i) q[i] = load_row<TX, 8, EXACT>(x + row * a.ldx, (i * LPR + l) * 8, C);
    };
    // past the last row the last one is read again (no branch around a load)
    load(min(r, a.N - 1));
    Params<KCH> weight, bias;
    weight.template init<LPR>(a.weight, 1.f, C, pw, l);
    bias.template init<LPR>(a.bias, 0.f, C, pb, l);
    if constexpr (KCH > 1) __syncthreads();
    // channels that wave w of a row holds
    auto count = [&](int w) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < KCH; ++i) n += max(0, min(C - (i * LPR + w * 64) * 8, (LPR < 64 ? LPR : 64) * 8));
        return float(n);
    };
    int slot = 0;

    for (; r < a.N; r += step) {
        // a wave's own mean and squared deviations around it, then the row's
        // from those: sum (x - mean)^2 = sum_w [Q_w + n_w (mean_w - mean)^2], as
        // safe against cancellation as two passes, with one barrier
        float v[KCH][8], sum = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const bool in = !EXACT || (i * LPR + l) * 8 < C;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = element(q[i], e);
                sum += in ? v[i][e] : 0.f;
            }
        }
        load(min(r + step, a.N - 1));
        constexpr int L = LPR < 64 ? LPR : 64;
        float mean = lane_sum<L>(sum) / fmaxf(count(l / 64), 1.f);
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int left = C - (i * LPR + l) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[i][e] - mean;
                sq += (EXACT ? 0 < left : e < left) ? d * d : 0.f;
            }
        }
        sq = lane_sum<L>(sq);
        if constexpr (WAVES > 1) {
            if ((threadIdx.x & 63) == 0) red[slot][l / 64] = float2{mean, sq};
            __syncthreads();
            float total = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) total += red[slot][w].x * count(w);
            mean = total / fc;
            sq = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const float d = red[slot][w].x - mean;
                sq += red[slot][w].y + count(w) * d * d;
            }
            slot ^= 1;                         // a wave that is ahead writes the other slot
        }
        const float rstd = 1.f / sqrtf(sq / fc + a.eps);
        Raw<TY, 8> out[KCH];
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            // lanes past the end work along and store nothing
            const int c = (i * LPR + l) * 8;
            float w[8], b[8];
            weight.template get<LPR>(i, w);
            bias.template get<LPR>(i, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = (v[i][e] - mean) * rstd * w[e] + b[e];
            if (a.drop.threshold) drop_chunk<EXACT>(r * C + c, a.drop, v[i]);
            out[i] = to_raw<TY, 8>(v[i]);
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) arrive(q[i]);
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8;
            store_row<EXACT>(y + r * a.ldo + c, C - c, out[i]);
        }
        if (l == 0 && a.mean) {
            a.mean[r] = mean;
            a.rstd[r] = rstd;
        }
    }
}

// rows wider than the largest group holds: one workgroup per row, three reads of it
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

template <typename TX, typename TY, int LPR, int KCH, bool EXACT>
__global__ __launch_bounds__(threads_of(LPR)) void norm_rows_bwd_kernel(const NormArgs a)
{
    constexpr int G = threads_of(LPR) / LPR;
    __shared__ float red[2][2][threads_of(LPR) / 64];
    __shared__ __align__(16) float part[LPR * KCH * 8];    // weight, then partial sums
    const int l = threadIdx.x % LPR, g = threadIdx.x / LPR, C = a.C;
    const TX *x = static_cast<const TX *>(a.x);
    const TY *dy = static_cast<const TY *>(a.dy);
    TX *dx = static_cast<TX *>(a.out);
    const float fc = float(C);
    const int64_t step = int64_t(gridDim.x) * G;
    int64_t r = int64_t(blockIdx.x) * G + g;

    float dw[KCH][8], db[KCH][8];
    Raw<TX, 8> xc[KCH], xn[KCH];
    Raw<TY, 8> yc[KCH], yn[KCH];
    float mc, rc, mn, rn;                              // mean and rstd of the rows in xc and xn
    auto load = [&](int64_t row, Raw<TX, 8> (&xp)[KCH], Raw<TY, 8> (&yp)[KCH], float &m, float &rs) {
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            xp[i] = load_row<TX, 8, EXACT>(x + row * a.ldx, (i * LPR + l) * 8, C);
            yp[i] = load_row<TY, 8, EXACT>(dy + row * a.ldy, (i * LPR + l) * 8, C);
        }
        m = a.mean[row];
        rs = a.rstd[row];
    };
    if (a.N > 0) load(min(r, a.N - 1), xc, yc, mc, rc);
    Params<KCH> weight;
    weight.template init<LPR>(a.weight, 1.f, C, part, l);
    if constexpr (KCH > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < KCH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;

    int slot = 0;
    for (; r < a.N; r += step) {
        load(min(r + step, a.N - 1), xn, yn, mn, rn);   // past the last row: the last one again
        float h[KCH][8], z[KCH][8], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8, left = C - c;
            float w[8];
            weight.template get<LPR>(i, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = element(yc[i], e);
            if (a.drop.threshold) drop_chunk<EXACT>(r * C + c, a.drop, z[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = EXACT ? 0 < left : e < left;
                h[i][e] = in ? (element(xc[i], e) - mc) * rc : 0.f;
                if (EXACT) z[i][e] = in ? z[i][e] : 0.f;
                dw[i][e] += z[i][e] * h[i][e];
                db[i][e] += z[i][e];
                z[i][e] *= w[e];
                s1 += z[i][e];
                s2 += z[i][e] * h[i][e];
            }
        }
        row_sum2<LPR>(s1, s2, red, slot);
        slot ^= 1;
        s1 /= fc;
        s2 /= fc;
        Raw<TX, 8> out[KCH];
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = rc * (z[i][e] - s1 - h[i][e] * s2);
            out[i] = to_raw<TX, 8>(z[i]);
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            xc[i] = xn[i];
            yc[i] = yn[i];
        }
        mc = mn;
        rc = rn;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8;
            store_row<EXACT>(dx + r * a.ldo + c, C - c, out[i]);
        }
    }

    if (!a.partial) return;
    // the workgroup's groups added in order, dweight first, then dbias
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        for (int q = 0; q < G; ++q) {
            __syncthreads();
            if (g == q)
#pragma unroll
                for (int i = 0; i < KCH; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float &t = part[(i * LPR + l) * 8 + e];
                        t = (q ? t : 0.f) + (k ? db[i][e] : dw[i][e]);
                    }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += threads_of(LPR))
            a.partial[(int64_t(blockIdx.x) * 2 + k) * C + c] = part[c];
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
    // the next columns' part[0] is written by the threads that read this one's
    for (int64_t k0 = int64_t(blockIdx.x) * 16; k0 < 2 * int64_t(C); k0 += int64_t(gridDim.x) * 16) {
        const int64_t k = k0 + col;
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
}

// The group that holds a row of C channels: as few lanes per row as keep it to
// one chunk each (so narrow rows fill whole waves), then one wave with several
// chunks per lane (no barrier per row), past that a workgroup. Backward a lane
// also keeps its share of dweight and dbias for every chunk, so the workgroup
// comes sooner. 4096 channels, bf16, 32768 rows: forward 122 us with one wave of
// 8 chunks, 127 with four of 2, 146 with eight of 1; backward 186, 166 and 171.
// lpr 0: no group holds it (the row is read again for each pass).
struct Group {
    int lpr, kch;
};
Group group_of(int64_t C, bool backward)
{
    const int64_t ch = (C + 7) / 8;
    if (C < 8) return {0, 0};
    if (ch <= 8) return {8, 1};
    if (ch <= 16) return {16, 1};
    if (ch <= 32) return {32, 1};
    if (ch <= 64) return {64, 1};
    if (ch <= 128) return {64, 2};
    if (ch <= 256) return backward ? Group{256, 1} : Group{64, 4};
    if (ch <= 512) return backward ? Group{256, 2} : Group{64, 8};
    if (ch <= 1024) return {256, 4};
    return {0, 0};
}

template <bool BACKWARD, typename F>
hipError_t with_group(const Group &g, F f)
{
    using std::integral_constant;
    const auto call = [&](auto lpr, auto kch) { return f(lpr, kch); };
#define IM2WIN_GROUP(L, K) \
    if (g.lpr == L && g.kch == K) return call(integral_constant<int, L>{}, integral_constant<int, K>{});
    IM2WIN_GROUP(8, 1)
    IM2WIN_GROUP(16, 1)
    IM2WIN_GROUP(32, 1)
    IM2WIN_GROUP(64, 1)
    IM2WIN_GROUP(64, 2)
    if constexpr (BACKWARD) {
        IM2WIN_GROUP(256, 1)
        IM2WIN_GROUP(256, 2)
    } else {
        IM2WIN_GROUP(64, 4)
        IM2WIN_GROUP(64, 8)
    }
    IM2WIN_GROUP(256, 4)
#undef IM2WIN_GROUP
    return hipErrorInvalidValue;
}

// Workgroups at most: forward as many as the CUs hold (one wave of 8 chunks: 12
// waves to a CU, 4 chunks: 20, else 32; 200000 rows of 256, bf16: 63.7, 46.1, 41.5 and
// 41.6 us with 512, 1024, 2048 and 4096); backward 8 waves to a CU, since each
// leaves a row of partial sums (12 and 16 waves measured slower). Rows read again:
// the same limit (4096 rows of 9001, bf16, forward 63.9 us; a workgroup for each row
// 57.2), and 32 parts of the rows for dweight and dbias, where few rows must not pay for
// many parts (backward 188, 148 and 132 us with 16, 32 and 64 parts; 500 rows of 20011,
// fp32: 52.1, 52.8 and 54.6).
constexpr int64_t kMaxBlocksFwd = 2048;
int64_t max_blocks_fwd(const Group &g) { return g.kch == 8 ? 768 : g.kch == 4 ? 1280 : kMaxBlocksFwd; }
int64_t max_blocks_bwd(const Group &g) { return 256 * 8 / (threads_of(g.lpr) / 64); }
constexpr int64_t kColSplits = 32;

}  // namespace

int64_t norm_rows_partials(int64_t N, int64_t C)
{
    const Group g = group_of(C, true);
    if (!g.lpr) return kColSplits;
    const int64_t per = threads_of(g.lpr) / g.lpr;
    return std::max<int64_t>(1, std::min((N + per - 1) / per, max_blocks_bwd(g)));
}

hipError_t launch_norm_rows_fwd(const NormArgs &a, hipStream_t s)
{
    const Group g = group_of(a.C, false);
    return with_norm_types(a.dtype, a.y_dtype, [&](auto tx, auto ty) {
        using TX = typename decltype(tx)::type;
        using TY = typename decltype(ty)::type;
        if (!g.lpr) {
            const dim3 grid(unsigned(std::min(a.N, kMaxBlocksFwd)));
            hipLaunchKernelGGL((norm_rows_fwd_wide_kernel<TX, TY>), grid, dim3(kThreads), 0, s, a);
            return hipGetLastError();
        }
        return with_group<false>(g, [&](auto lpr, auto kch) {
            constexpr int LPR = decltype(lpr)::value, KCH = decltype(kch)::value;
            const int64_t per = threads_of(LPR) / LPR;
            const dim3 grid(unsigned(std::min((a.N + per - 1) / per, max_blocks_fwd(g))));
            if (a.C % 8 == 0)
                hipLaunchKernelGGL((norm_rows_fwd_kernel<TX, TY, LPR, KCH, true>), grid, dim3(threads_of(LPR)), 0, s,
                                   a);
            else
                hipLaunchKernelGGL((norm_rows_fwd_kernel<TX, TY, LPR, KCH, false>), grid, dim3(threads_of(LPR)), 0, s,
                                   a);
            return hipGetLastError();
        });
    });
}

hipError_t launch_norm_rows_bwd(const NormArgs &a, hipStream_t s)
{
    const Group g = group_of(a.C, true);
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
        return with_group<true>(g, [&](auto lpr, auto kch) {
            constexpr int LPR = decltype(lpr)::value, KCH = decltype(kch)::value;
            const dim3 grid{unsigned(blocks)};
            if (a.C % 8 == 0)
                hipLaunchKernelGGL((norm_rows_bwd_kernel<TX, TY, LPR, KCH, true>), grid, dim3(threads_of(LPR)), 0, s,
                                   a);
            else
                hipLaunchKernelGGL((norm_rows_bwd_kernel<TX, TY, LPR, KCH, false>), grid, dim3(threads_of(LPR)), 0, s,
                                   a);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || !a.partial) return e;
    return launch_norm_reduce(a.partial, blocks, a.C, a.dweight, a.dbias, s);
}

hipError_t launch_norm_reduce(const float *partial, int64_t rows, int C, float *dweight, float *dbias,
                              hipStream_t s)
{
    const int64_t groups = std::min((2 * int64_t(C) + 15) / 16, max_groups(1024));
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(unsigned(groups)), dim3(1024), 0, s, partial, int(rows), C, dweight,
                       dbias);
    return hipGetLastError();
}

}  // namespace im2win
