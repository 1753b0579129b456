// The norm after a block, its gate, the residual sum and the norm before the next
// block (im2win_block.h) over rows of channels: forward, backward and the reduction of
// the parameters' gradients. All bound by HBM: forward reads b and r and writes out and
// y once, backward reads dy, dout, b and out and writes dr and db once.
//
// A row of each tensor is held in registers by a group of LPR lanes, KCH chunks of 8
// channels per lane, between the two norms as well; the next row's loads are issued
// before the current row is worked on. A workgroup takes consecutive rows, so that the
// gate stays in registers until its group ends.
//
// Backward needs, per gate's group and channel, S1 = sum t xhat(b) and S2 = sum t alone:
//   dgate = bs (pw S1 + pb S2),  dpw = sum_groups bs gate S1,  dpb = sum_groups bs gate S2
// (without the norm after the block S1 = sum t b and dgate = bs S1), and of the next
// norm sum dy xhat(out) and sum dy: four sums per channel stay in registers over all of a
// workgroup's rows. S1 and S2 leave at the end of each group that the workgroup sees,
// the others at its end; a second launch adds them in a fixed order.
// Rows of more than 8192 channels are wider than a group holds and are read again for each
// pass over them.
// 32768 rows of 4096, bf16: forward 212 us (5.1 TB/s), backward 317 and 10 for the second
// launch (4.9). 19941 rows of 1001, fp32 with fp16, a gate for every 289: 82 and 9 (4.0).
// From 4097 channels on backward is no longer bound by HBM: with two chunks to each of 512
// lanes 56 to 238 registers do not fit and go through scratch memory (8192 rows of 8192, bf16:
// forward 115 us, 4.7 TB/s, backward 196, 4.1; fp32 217 and 533; 8192 rows of 8200 235 and 519).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../block_launch.hpp"
#include "norm_common.hpp"

namespace im2win {
namespace {

constexpr int kThreads = 256;
constexpr int threads_of(int lpr) { return lpr > 64 ? lpr : kThreads; }

// Rows of block b of B: consecutive. Record (block, group of gates) is number
// block + group: blocks share at most their end's group, so no two are the same. Where a
// block ends with a group, the number after its last record is no one's: that block
// writes zeros there, so that records 0 .. B + groups - 2 are all written.
__host__ __device__ __forceinline__ int64_t first_row(int64_t N, int64_t B, int64_t b)
{
    const int64_t q = N / B, rem = N - q * B;
    return q * b + (b < rem ? b : rem);
}
__device__ __forceinline__ int block_of(uint32_t N, uint32_t B, uint32_t row)
{
    const uint32_t q = N / B, rem = N - q * B;             // B <= N: q >= 1
    return int(row < rem * (q + 1) ? row / (q + 1) : rem + (row - rem * (q + 1)) / q);
}

// sum of (a, b) over the LPR lanes of a row; `slot` alternates between calls
template <int LPR>
__device__ __forceinline__ void row_sum2(float &a, float &b, float2 (*red)[threads_of(LPR) / 64], int &slot)
{
    a = lane_sum<(LPR < 64 ? LPR : 64)>(a);
    b = lane_sum<(LPR < 64 ? LPR : 64)>(b);
    if constexpr (LPR > 64) {
        if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = float2{a, b};
        __syncthreads();
        a = 0.f;
        b = 0.f;
#pragma unroll
        for (int w = 0; w < LPR / 64; ++w) {
            a += red[slot][w].x;
            b += red[slot][w].y;
        }
        slot ^= 1;
    }
}

// channels of a row that wave w of its lanes holds
template <int LPR, int KCH>
__device__ __forceinline__ float count_of(int C, int w)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < KCH; ++i) n += max(0, min(C - (i * LPR + w * 64) * 8, (LPR < 64 ? LPR : 64) * 8));
    return float(n);
}

// Mean (0 but for layer norms) and rstd of a row: each wave's own mean and squared
// deviations around it, then the row's from those: sum (z - mean)^2 = sum_w [Q_w + n_w
// (mean_w - mean)^2], as safe against cancellation as two passes, with one barrier.
template <int LPR, int KCH>
__device__ __forceinline__ float2 row_stats(const float (&v)[KCH][8], int l, int C, int layer, float eps,
                                            float2 (*red)[threads_of(LPR) / 64], int &slot)
{
    constexpr int L = LPR < 64 ? LPR : 64, WAVES = LPR > 64 ? LPR / 64 : 1;
    const float fc = float(C);
    float mean = 0.f, sq = 0.f;
    if (layer) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += (i * LPR + l) * 8 + e < C ? v[i][e] : 0.f;
        mean = lane_sum<L>(sum) / fmaxf(count_of<LPR, KCH>(C, l / 64), 1.f);
    }
#pragma unroll
    for (int i = 0; i < KCH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = v[i][e] - mean;
            sq += (i * LPR + l) * 8 + e < C ? d * d : 0.f;
        }
    sq = lane_sum<L>(sq);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) red[slot][l / 64] = float2{mean, sq};
        __syncthreads();
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) total += red[slot][w].x * count_of<LPR, KCH>(C, w);
        mean = total / fc;
        sq = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float d = red[slot][w].x - mean;
            sq += red[slot][w].y + count_of<LPR, KCH>(C, w) * d * d;
        }
        slot ^= 1;
    }
    return float2{mean, 1.f / sqrtf(sq / fc + eps)};
}

// channels c .. c + 7 of a parameter vector, `absent` where there is none
__device__ __forceinline__ void param(const float *p, float absent, int c, int C, float (&f)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = absent;
    if (p) load_some<8>(p + c, max(0, C - c), f);
}

// channels c .. c + 7 of a row of C, zeros past its end (EXACT: anything), without a branch.
// A lane that holds a whole row (C < 8) reads its elements one by one.
template <int LPR, bool EXACT, typename T>
__device__ __forceinline__ Raw<T, 8> load_chunk(const T *row, int c, int C)
{
    if constexpr (LPR == 1) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = float(row[min(e, C - 1)]);
#pragma unroll
        for (int e = 1; e < 8; ++e) f[e] = e < C ? f[e] : 0.f;
        return to_raw<T, 8>(f);
    } else {
        return load_row<T, 8, EXACT>(row, c, C);
    }
}

template <bool EXACT, typename T>
__device__ __forceinline__ void store_row(T *p, int left, const Raw<T, 8> &r)
{
    if constexpr (EXACT) {
        if (left > 0) store_raw(p, r);
    } else {
        store_some_raw(p, max(left, 0), r);
    }
}

template <typename TR, typename TB, int LPR, int KCH, bool EXACT>
__global__ __launch_bounds__(threads_of(LPR)) void res_norm_fwd_kernel(const ResNormArgs a)
{
    constexpr int G = threads_of(LPR) / LPR;               // rows in flight per workgroup
    __shared__ float2 red[2][threads_of(LPR) / 64];
    const int l = threadIdx.x % LPR, C = a.C;
    const TB *b = static_cast<const TB *>(a.b);
    const TR *r = static_cast<const TR *>(a.r);
    const int64_t end = first_row(a.N, gridDim.x, blockIdx.x + 1);
    int64_t row = first_row(a.N, gridDim.x, blockIdx.x) + threadIdx.x / LPR;

    Raw<TB, 8> qb[KCH];
    Raw<TR, 8> qr[KCH];
    auto load = [&](int64_t k) {
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            qb[i] = load_chunk<LPR, EXACT>(b + k * a.ldb, (i * LPR + l) * 8, C);
            qr[i] = load_chunk<LPR, EXACT>(r + k * a.ldr, (i * LPR + l) * 8, C);
        }
    };
    // past the last row that one is read again (no branch around a load)
    load(min(row, a.N - 1));
    float pw[KCH][8], pb[KCH][8], w[KCH][8], bias[KCH][8], gate[KCH][8];
#pragma unroll
    for (int i = 0; i < KCH; ++i) {
        const int c = (i * LPR + l) * 8;
        param(a.pw, 1.f, c, C, pw[i]);
        param(a.pb, 0.f, c, C, pb[i]);
        param(a.w, 1.f, c, C, w[i]);
        param(a.bias, 0.f, c, C, bias[i]);
    }
    int64_t group = -1;
    int slot = 0;
    // a workgroup-wide row's barriers: every thread makes the same number of rounds
    for (; row < end; row += G) {
        const int64_t g = a.groups > 1 ? row / a.rows : 0;
        if (g != group) {
            group = g;
#pragma unroll
            for (int i = 0; i < KCH; ++i) {
                param(a.gate ? a.gate + g * C : nullptr, 1.f, (i * LPR + l) * 8, C, gate[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) gate[i][e] *= a.bs;
            }
        }
        float v[KCH][8], o[KCH][8];
#pragma unroll
        for (int i = 0; i < KCH; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = element(qb[i], e);
                o[i][e] = element(qr[i], e);
            }
        load(min(row + G, a.N - 1));
        float2 st{0.f, 0.f};
        if (a.post) {
            st = row_stats<LPR, KCH>(v, l, C, a.layer, a.eps, red, slot);
#pragma unroll
            for (int i = 0; i < KCH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = (v[i][e] - st.x) * st.y * pw[i][e] + pb[i][e];
        }
        Raw<TR, 8> out[KCH];
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[i][e] = a.rs * o[i][e] + gate[i][e] * v[i][e];
            out[i] = to_raw<TR, 8>(o[i]);
        }
        const float2 so = row_stats<LPR, KCH>(o, l, C, a.layer, a.eps, red, slot);
        Raw<TB, 8> y[KCH];
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[i][e] = (o[i][e] - so.x) * so.y * w[i][e] + bias[i][e];
            y[i] = to_raw<TB, 8>(o[i]);
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            arrive(qb[i]);
            arrive(qr[i]);
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8;
            store_row<EXACT>(static_cast<TR *>(a.out) + row * a.ldo + c, C - c, out[i]);
            store_row<EXACT>(static_cast<TB *>(a.y) + row * a.ldy + c, C - c, y[i]);
        }
        if (l == 0 && a.stats) reinterpret_cast<float4 *>(a.stats)[row] = float4{st.x, st.y, so.x, so.y};
    }
}

// any row: one workgroup per row, which reads it again for each pass
template <typename TR, typename TB>
__global__ __launch_bounds__(kThreads) void res_norm_fwd_wide_kernel(const ResNormArgs a)
{
    __shared__ float2 red[2][kThreads / 64];
    const int C = a.C;
    const float fc = float(C);
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const TB *b = static_cast<const TB *>(a.b) + row * a.ldb;
        const TR *r = static_cast<const TR *>(a.r) + row * a.ldr;
        const float *gate = a.gate ? a.gate + (a.groups > 1 ? row / a.rows : 0) * C : nullptr;
        float v[8], zero = 0.f;
        float2 st{0.f, 0.f}, so{0.f, 0.f};
        if (a.post) {
            if (a.layer) {
                float sum = 0.f;
                for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
                    load_some<8>(b + c, C - c, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum += v[e];
                }
                row_sum2<kThreads>(sum, zero, red, slot);
                st.x = sum / fc;
            }
            float sq = 0.f;
            for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
                load_some<8>(b + c, C - c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sq += e < C - c ? (v[e] - st.x) * (v[e] - st.x) : 0.f;
            }
            row_sum2<kThreads>(sq, zero, red, slot);
            st.y = 1.f / sqrtf(sq / fc + a.eps);
        }
        auto sum_at = [&](int c, float (&o)[8]) {
            float p[8], q[8];
            load_some<8>(b + c, C - c, v);
            load_some<8>(r + c, C - c, o);
            if (a.post) {
                param(a.pw, 1.f, c, C, p);
                param(a.pb, 0.f, c, C, q);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (v[e] - st.x) * st.y * p[e] + q[e];
            }
            param(gate, 1.f, c, C, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = e < C - c ? a.rs * o[e] + p[e] * a.bs * v[e] : 0.f;
        };
        float o[8];
        if (a.layer) {
            float sum = 0.f;
            for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
                sum_at(c, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += o[e];
            }
            row_sum2<kThreads>(sum, zero, red, slot);
            so.x = sum / fc;
        }
        float sq = 0.f;
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            sum_at(c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) sq += e < C - c ? (o[e] - so.x) * (o[e] - so.x) : 0.f;
        }
        row_sum2<kThreads>(sq, zero, red, slot);
        so.y = 1.f / sqrtf(sq / fc + a.eps);
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            float w[8], bias[8];
            sum_at(c, o);
            store_some<8>(static_cast<TR *>(a.out) + row * a.ldo + c, C - c, o);
            param(a.w, 1.f, c, C, w);
            param(a.bias, 0.f, c, C, bias);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (o[e] - so.x) * so.y * w[e] + bias[e];
            store_some<8>(static_cast<TB *>(a.y) + row * a.ldy + c, C - c, o);
        }
        if (threadIdx.x == 0 && a.stats)
            reinterpret_cast<float4 *>(a.stats)[row] = float4{st.x, st.y, so.x, so.y};
    }
}

// Workspace of the backward pass: the blocks' sums of the next norm [B][2][C], then
// the records [B + groups][2][C] and their groups, then (wide rows) each row's two
// means [N][2]. Where lanes take whole groups there are B records and nothing after them.
struct Sums {
    float *norm, *record;
    int *group;
    float2 *means;
};
__host__ __device__ __forceinline__ Sums sums_of(const ResNormArgs &a, int64_t B)
{
    float *p = static_cast<float *>(a.ws);
    const int64_t G = a.groups > 1 ? a.groups : 1;
    float *end = p + (2 * B + G) * 2 * a.C;
    return {p, p + B * 2 * a.C, reinterpret_cast<int *>(end), reinterpret_cast<float2 *>(end + (B + G + 1) / 2 * 2)};
}

template <int THREADS>
__device__ __forceinline__ void skip_record(const Sums &sums, int64_t k, int C)
{
    for (int c = threadIdx.x; c < 2 * C; c += THREADS) sums.record[k * 2 * C + c] = 0.f;
    if (threadIdx.x == 0) sums.group[k] = 0;
}

// OWN: short groups of rows with a gate each. A row's lanes take whole groups, so that
// dgate leaves from their registers and dpw and dpb stay there like the next norm's sums.
template <typename TR, typename TB, int LPR, int KCH, bool EXACT, bool OWN>
__global__ __launch_bounds__(threads_of(LPR)) void res_norm_bwd_kernel(const ResNormArgs a)
{
    constexpr int THREADS = threads_of(LPR), G = THREADS / LPR;
    __shared__ float2 red[2][THREADS / 64];
    __shared__ __align__(16) float part[LPR == 1 ? THREADS / 8 : LPR * KCH * 8];
    const int l = threadIdx.x % LPR, q = threadIdx.x / LPR, C = a.C;
    const float fc = float(C);
    const TB *dy = static_cast<const TB *>(a.dy), *b = static_cast<const TB *>(a.b);
    const TR *dout = static_cast<const TR *>(a.dout), *out = static_cast<const TR *>(a.out);
    const float4 *stats = reinterpret_cast<const float4 *>(a.stats);
    const int64_t begin = first_row(a.N, gridDim.x, blockIdx.x), end = first_row(a.N, gridDim.x, blockIdx.x + 1);
    const Sums sums = sums_of(a, gridDim.x);
    const bool records = a.ws && (a.post || a.gate), has_dout = a.dout != nullptr;

    Raw<TB, 8> qy[KCH], qb[KCH], ny[KCH], nb[KCH];
    Raw<TR, 8> qd[KCH], qo[KCH], nd[KCH], no[KCH];
    float4 qs, ns;
    auto load = [&](int64_t k, Raw<TB, 8> (&y)[KCH], Raw<TB, 8> (&x)[KCH], Raw<TR, 8> (&d)[KCH], Raw<TR, 8> (&o)[KCH],
                    float4 &s) {
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8;
            y[i] = load_chunk<LPR, EXACT>(dy + k * a.lddy, c, C);
            x[i] = load_chunk<LPR, EXACT>(b + k * a.ldb, c, C);
            o[i] = load_chunk<LPR, EXACT>(out + k * a.ldo, c, C);
            // without a dout: out again, and cleared below
            d[i] = load_chunk<LPR, EXACT>(has_dout ? dout + k * a.lddo : out + k * a.ldo, c, C);
        }
        s = stats[k];
    };
    float w[KCH][8], gq[KCH][8], s1[KCH][8], s2[KCH][8], s3[KCH][8], s4[KCH][8];
#pragma unroll
    for (int i = 0; i < KCH; ++i) {
        param(a.w, 1.f, (i * LPR + l) * 8, C, w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s3[i][e] = s4[i][e] = 0.f;
    }
    // the workgroup's groups of lanes added in order into dst[C]
    auto flush = [&](const float (&v)[KCH][8], float *dst) {
        if constexpr (LPR == 1) {              // a lane's row: first over the waves
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = lane_sum<64>(v[0][e]);
                if ((threadIdx.x & 63) == 0) part[(threadIdx.x >> 6) * 8 + e] = t;
            }
            __syncthreads();
            if (int(threadIdx.x) < C)
                dst[threadIdx.x] = (part[threadIdx.x] + part[8 + threadIdx.x]) + (part[16 + threadIdx.x] + part[24 + threadIdx.x]);
            return;
        }
        for (int k = 0; k < G; ++k) {
            __syncthreads();
            if (q == k)
#pragma unroll
                for (int i = 0; i < KCH; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float &t = part[(i * LPR + l) * 8 + e];
                        t = (k ? t : 0.f) + v[i][e];
                    }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += THREADS) dst[c] = part[c];
    };
    int slot = 0;
    // the row that is in q*; `valid`: it is one of this lane's
    const auto work = [&](int64_t row, bool valid) {
        float t[KCH][8], h[KCH][8], u = 0.f, v = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int left = valid ? C - (i * LPR + l) * 8 : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = EXACT ? 0 < left : e < left;
                const float y = in ? element(qy[i], e) : 0.f;
                h[i][e] = in ? (element(qo[i], e) - qs.z) * qs.w : 0.f;
                s3[i][e] += y * h[i][e];
                s4[i][e] += y;
                t[i][e] = y * w[i][e];
                u += t[i][e];
                v += t[i][e] * h[i][e];
            }
        }
        row_sum2<LPR>(u, v, red, slot);
        u = a.layer ? u / fc : 0.f;
        v /= fc;
        Raw<TR, 8> dr[KCH];
        Raw<TB, 8> db[KCH];
        float m = 0.f, n = 0.f;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int left = valid ? C - (i * LPR + l) * 8 : 0;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = EXACT ? 0 < left : e < left;
                t[i][e] = (has_dout ? element(qd[i], e) : 0.f) + qs.w * (t[i][e] - u - h[i][e] * v);
                t[i][e] = in ? t[i][e] : 0.f;
                f[e] = a.rs * t[i][e];
                const float x = in ? element(qb[i], e) : 0.f;
                h[i][e] = a.post ? (in ? (x - qs.x) * qs.y : 0.f) : x;
                s1[i][e] += t[i][e] * h[i][e];
                s2[i][e] += t[i][e];
                t[i][e] *= gq[i][e];
                m += t[i][e];
                n += t[i][e] * h[i][e];
            }
            dr[i] = to_raw<TR, 8>(f);
        }
        if (a.post) {
            row_sum2<LPR>(m, n, red, slot);
            m = a.layer ? m / fc : 0.f;
            n /= fc;
#pragma unroll
            for (int i = 0; i < KCH; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) t[i][e] = qs.y * (t[i][e] - m - h[i][e] * n);
        }
#pragma unroll
        for (int i = 0; i < KCH; ++i) db[i] = to_raw<TB, 8>(t[i]);
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            qy[i] = ny[i];
            qb[i] = nb[i];
            qd[i] = nd[i];
            qo[i] = no[i];
        }
        qs = ns;
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            const int c = (i * LPR + l) * 8, left = valid ? C - c : 0;
            store_row<EXACT>(static_cast<TR *>(a.dr) + row * a.lddr + c, left, dr[i]);
            store_row<EXACT>(static_cast<TB *>(a.db) + row * a.lddb + c, left, db[i]);
        }
    };
    // gq = gate post_weight branch_scale, and the group's sums cleared
    const auto start = [&](const float (&gate)[KCH][8]) {
#pragma unroll
        for (int i = 0; i < KCH; ++i) {
            float p[8];
            param(a.post ? a.pw : nullptr, 1.f, (i * LPR + l) * 8, C, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                gq[i][e] = gate[i][e] * (a.bs * p[e]);
                s1[i][e] = s2[i][e] = 0.f;
            }
        }
    };
    const auto gate_of = [&](int64_t g, float (&gate)[KCH][8]) {
#pragma unroll
        for (int i = 0; i < KCH; ++i) param(a.gate ? a.gate + g * C : nullptr, 1.f, (i * LPR + l) * 8, C, gate[i]);
    };
    if constexpr (OWN) {
        const int64_t units = int64_t(gridDim.x) * G, unit = int64_t(blockIdx.x) * G + q;
        int64_t g = first_row(a.groups, units, unit);
        const int64_t last = first_row(a.groups, units, unit + 1), rounds = (a.groups + units - 1) / units;
        float gate[KCH][8], next[KCH][8], p1[KCH][8] = {}, p2[KCH][8] = {};
        load(min(g * a.rows, a.N - 1), qy, qb, qd, qo, qs);
        gate_of(min(g, a.groups - 1), gate);
        // every lane makes the same number of rounds
        for (int64_t round = 0; round < rounds; ++round, ++g) {
            const bool valid = g < last;
            start(gate);
            for (int64_t r = 0; r < a.rows; ++r) {
                const int64_t row = g * a.rows + r;
                load(min(row + 1, a.N - 1), ny, nb, nd, no, ns);
                if (r + 1 == a.rows) gate_of(min(g + 1, a.groups - 1), next);
                work(row, valid);
            }
#pragma unroll
            for (int i = 0; i < KCH; ++i) {
                const int c = (i * LPR + l) * 8;
                float pw[8], pb[8], d[8];
                param(a.post ? a.pw : nullptr, 1.f, c, C, pw);
                param(a.post ? a.pb : nullptr, 0.f, c, C, pb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p1[i][e] += gate[i][e] * s1[i][e];
                    p2[i][e] += gate[i][e] * s2[i][e];
                    d[e] = a.bs * (pw[e] * s1[i][e] + pb[e] * s2[i][e]);
                    gate[i][e] = next[i][e];
                }
                if (a.dgate && valid) store_some<8>(a.dgate + g * C + c, max(C - c, 0), d);
            }
        }
        if (records) {                         // (branch_scale is the second launch's)
            flush(p1, sums.record + int64_t(blockIdx.x) * 2 * C);
            flush(p2, sums.record + (int64_t(blockIdx.x) * 2 + 1) * C);
        }
    } else {
        for (int64_t from = begin; from < end;) {
            // the rows of one gate
            const int64_t g = a.groups > 1 ? from / a.rows : 0;
            const int64_t to = a.groups > 1 ? min(end, (g + 1) * a.rows) : end;
            float gate[KCH][8];
            gate_of(g, gate);
            start(gate);
            load(min(from + q, a.N - 1), qy, qb, qd, qo, qs);
            for (int64_t row = from + q; row < to; row += G) {
                load(min(row + G, a.N - 1), ny, nb, nd, no, ns);
                work(row, true);
            }
            if (records) {
                float *rec = sums.record + (blockIdx.x + g) * 2 * C;
                flush(s1, rec);
                flush(s2, rec + C);
                if (threadIdx.x == 0) sums.group[blockIdx.x + g] = int(g);
                if (to == end && a.groups > 1 && end % a.rows == 0 && end < a.N) skip_record<THREADS>(sums, blockIdx.x + g + 1, C);
            }
            from = to;
        }
    }
    if (!a.ws) return;
    flush(s3, sums.norm + int64_t(blockIdx.x) * 2 * C);
    flush(s4, sums.norm + (int64_t(blockIdx.x) * 2 + 1) * C);
}

// any row: one workgroup per row, three reads of it
template <typename TR, typename TB>
__global__ __launch_bounds__(kThreads) void res_norm_bwd_wide_kernel(const ResNormArgs a, float2 *means)
{
    __shared__ float2 red[2][kThreads / 64];
    const int C = a.C;
    const float fc = float(C);
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const TB *dy = static_cast<const TB *>(a.dy) + row * a.lddy, *b = static_cast<const TB *>(a.b) + row * a.ldb;
        const TR *dout = a.dout ? static_cast<const TR *>(a.dout) + row * a.lddo : nullptr;
        const TR *out = static_cast<const TR *>(a.out) + row * a.ldo;
        const float *gate = a.gate ? a.gate + (a.groups > 1 ? row / a.rows : 0) * C : nullptr;
        const float4 st = reinterpret_cast<const float4 *>(a.stats)[row];
        float h[8], g[8], w[8], u = 0.f, v = 0.f;
        auto next = [&](int c) {               // xhat(out) and dy * weight
            load_some<8>(out + c, C - c, h);
            load_some<8>(dy + c, C - c, g);
            param(a.w, 1.f, c, C, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = e < C - c ? (h[e] - st.z) * st.w : 0.f;
                g[e] *= w[e];
            }
        };
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            next(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u += g[e];
                v += g[e] * h[e];
            }
        }
        row_sum2<kThreads>(u, v, red, slot);
        u = a.layer ? u / fc : 0.f;
        v /= fc;
        if (means && threadIdx.x == 0) means[row] = float2{u, v};
        float t[8], m = 0.f, n = 0.f;
        auto through = [&](int c) {            // t, then xhat(b) (or b) in h
            next(c);
            float d[8] = {};
            if (dout) load_some<8>(dout + c, C - c, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = e < C - c ? d[e] + st.w * (g[e] - u - h[e] * v) : 0.f;
            load_some<8>(b + c, C - c, h);
            if (a.post)
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = e < C - c ? (h[e] - st.x) * st.y : 0.f;
        };
        auto gated = [&](int c) {
            float p[8];
            param(gate, 1.f, c, C, w);
            param(a.post ? a.pw : nullptr, 1.f, c, C, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] *= w[e] * (a.bs * p[e]);
        };
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            through(c);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = a.rs * t[e];
            store_some<8>(static_cast<TR *>(a.dr) + row * a.lddr + c, C - c, f);
            gated(c);
            if (a.post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    m += t[e];
                    n += t[e] * h[e];
                }
            } else {
                store_some<8>(static_cast<TB *>(a.db) + row * a.lddb + c, C - c, t);
            }
        }
        if (!a.post) continue;
        row_sum2<kThreads>(m, n, red, slot);
        m = a.layer ? m / fc : 0.f;
        n /= fc;
        for (int c = threadIdx.x * 8; c < C; c += kThreads * 8) {
            through(c);
            gated(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = st.y * (t[e] - m - h[e] * n);
            store_some<8>(static_cast<TB *>(a.db) + row * a.lddb + c, C - c, t);
        }
    }
}

// the wide rows' sums: a workgroup takes 512 channels of one block's rows, a wave one
// row at a time
template <typename TR, typename TB>
__global__ __launch_bounds__(kThreads) void res_norm_cols_kernel(const ResNormArgs a)
{
    __shared__ float part[4][512];
    const int C = a.C, wave = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t B = gridDim.y, begin = first_row(a.N, B, blockIdx.y), end = first_row(a.N, B, blockIdx.y + 1);
    const int c0 = blockIdx.x * 512, c = c0 + l * 8, left = C - c;
    const Sums sums = sums_of(a, B);
    float w[8], s3[8] = {}, s4[8] = {};
    param(a.w, 1.f, c, C, w);
    auto flush = [&](const float (&v)[8], float *dst) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) part[wave][l * 8 + e] = v[e];
        __syncthreads();
        for (int i = threadIdx.x; i < 512 && c0 + i < C; i += kThreads)
            dst[c0 + i] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
    };
    for (int64_t from = begin; from < end;) {
        const int64_t g = a.groups > 1 ? from / a.rows : 0;
        const int64_t to = a.groups > 1 ? min(end, (g + 1) * a.rows) : end;
        float s1[8] = {}, s2[8] = {};
        if (left > 0)
            for (int64_t row = from + wave; row < to; row += 4) {
                const float4 st = reinterpret_cast<const float4 *>(a.stats)[row];
                const float2 mean = sums.means[row];
                float o[8], y[8], d[8] = {}, b[8];
                load_some<8>(static_cast<const TR *>(a.out) + row * a.ldo + c, left, o);
                load_some<8>(static_cast<const TB *>(a.dy) + row * a.lddy + c, left, y);
                load_some<8>(static_cast<const TB *>(a.b) + row * a.ldb + c, left, b);
                if (a.dout) load_some<8>(static_cast<const TR *>(a.dout) + row * a.lddo + c, left, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float h = (o[e] - st.z) * st.w;
                    const float t = d[e] + st.w * (y[e] * w[e] - mean.x - h * mean.y);
                    s3[e] += y[e] * h;
                    s4[e] += y[e];
                    s1[e] += t * (a.post ? (b[e] - st.x) * st.y : b[e]);
                    s2[e] += t;
                }
            }
        if (a.post || a.gate) {
            float *rec = sums.record + (blockIdx.y + g) * 2 * C;
            flush(s1, rec);
            flush(s2, rec + C);
            // every workgroup of the block's rows writes the same
            if (threadIdx.x == 0) sums.group[blockIdx.y + g] = int(g);
            if (to == end && a.groups > 1 && end % a.rows == 0 && end < a.N) skip_record<kThreads>(sums, blockIdx.y + g + 1, C);
        }
        from = to;
    }
    flush(s3, sums.norm + int64_t(blockIdx.y) * 2 * C);
    flush(s4, sums.norm + (int64_t(blockIdx.y) * 2 + 1) * C);
}

// Channels of a workgroup of the join, with 1024 threads: many threads a channel where
// there are few channels (4096 channels, 256 blocks: 15 us with 16, 9 with 64; 1001: 8
// with 16).
__host__ __device__ __forceinline__ int join_channels(int C) { return C >= 2048 ? 64 : 16; }
// Whether dgate's groups have few records each: 4 threads a channel then.
__host__ __device__ __forceinline__ bool short_groups(int64_t B, int64_t G) { return (B + G) / G <= 32; }

// The parameters' gradients from the blocks' sums: a workgroup takes 16 or 64
// channels of (dweight, dbias), of (dpw, dpb) or of one group's dgate, or 256 elements of
// the dgate of short groups.
__global__ __launch_bounds__(1024) void res_norm_join_kernel(const ResNormArgs a, int64_t B)
{
    __shared__ float2 part[1024];
    const int C = a.C, t = threadIdx.x;
    const Sums sums = sums_of(a, B);
    const int W = join_channels(C);
    const int64_t G = a.groups > 1 ? a.groups : 1, tiles = (C + W - 1) / W;
    const bool few = a.dgate && short_groups(B, G);
    const int64_t trees = (a.dgate && !few ? 2 + G : 2) * tiles, all = trees + (few ? (G * C + 255) / 256 : 0);
    const auto records = [&](int64_t g, int &first, int &last) {
        first = 0;
        last = int(B) - 1;
        if (a.groups > 1) {
            first = block_of(uint32_t(a.N), uint32_t(B), uint32_t(g * a.rows));
            last = block_of(uint32_t(a.N), uint32_t(B), uint32_t((g + 1) * a.rows - 1));
        }
    };
    for (int64_t k = blockIdx.x; k < all; k += gridDim.x) {
        // the channel, its job (0, 1, or 2 + group) and this thread's share of it
        const int64_t job = k < trees ? k / tiles : 2, e = (k - trees) * 256 + (t & 255);
        int64_t g = job - 2;
        int c = int(k - job * tiles) * W + t % W, q = t / W, Q = 1024 / W;
        if (k >= trees) {
            g = e / C;
            c = g < G ? int(e - g * C) : C;
            q = t >> 8;
            Q = 4;
        }
        float x = 0.f, y = 0.f;
        if (c < C) {
            if (job == 0 && (a.dw || a.dbias)) {
#pragma unroll 4
                for (int64_t b = q; b < B; b += Q) {
                    x += sums.norm[b * 2 * C + c];
                    y += sums.norm[(b * 2 + 1) * C + c];
                }
            } else if (job == 1 && (a.dpw || a.dpb)) {
#pragma unroll 4
                for (int64_t r = q; r < B + G - 1; r += Q) {
                    const float s = a.gate ? a.bs * a.gate[int64_t(sums.group[r]) * C + c] : a.bs;
                    x += s * sums.record[r * 2 * C + c];
                    y += s * sums.record[(r * 2 + 1) * C + c];
                }
            } else if (job >= 2) {
                int first, last;
                records(g, first, last);
#pragma unroll 4
                for (int64_t b = first + q; b <= last; b += Q) {
                    x += sums.record[(b + g) * 2 * C + c];
                    y += sums.record[((b + g) * 2 + 1) * C + c];
                }
            }
        }
        part[t] = float2{x, y};
        __syncthreads();
        const int width = 1024 / Q;            // threads of one share
        for (int m = Q / 2; m > 0; m >>= 1) {
            if (q < m) {
                part[t].x += part[t + m * width].x;
                part[t].y += part[t + m * width].y;
            }
            __syncthreads();
        }
        // the next job's part[t] is written by the threads that read this one's
        if (q > 0 || c >= C) continue;
        const float2 s = part[t];
        if (job == 0) {
            if (a.dw) a.dw[c] = s.x;
            if (a.dbias) a.dbias[c] = s.y;
        } else if (job == 1) {
            if (a.dpw) a.dpw[c] = s.x;
            if (a.dpb) a.dpb[c] = s.y;
        } else {
            const float pw = a.pw ? a.pw[c] : 1.f, pb = a.pb ? a.pb[c] : 0.f;
            a.dgate[g * C + c] = a.bs * (a.post ? pw * s.x + pb * s.y : s.x);
        }
    }
}

// no rows: the sums are 0
__global__ __launch_bounds__(kThreads) void res_norm_zero_kernel(const ResNormArgs a)
{
    const int64_t step = int64_t(gridDim.x) * kThreads;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < a.groups * a.C || i < a.C; i += step) {
        if (a.dgate && i < a.groups * a.C) a.dgate[i] = 0.f;
        if (i >= a.C) continue;
        for (float *p : {a.dpw, a.dpb, a.dw, a.dbias})
            if (p) p[i] = 0.f;
    }
}

// The group that holds a row of C channels: as few lanes as keep it to one chunk each,
// then two chunks a lane: fewer waves meet at a row's barriers, and backward one wave to a
// row needs none. us of 256 (lanes, chunks) measured with 8 workgroups' worth of waves and
// more: 32768 rows of 4096, bf16, forward (256, 2) 214, (512, 1) 221 .. 284, (128, 4) 215;
// backward 329, 325 and -; 19941 rows of 1001, fp32 with fp16, backward (64, 2) 103, (128, 1)
// 133, forward 59.5 and 56.5; 65536 rows of 2048, bf16, backward (256, 1) 337, (128, 2) 358.
// (512, 2) is there for the rows that (256, 2) does not hold.
// lpr 0: no group holds it.
struct Group {
    int lpr, kch;
};
Group group_of(int64_t C, bool backward)
{
    const int64_t ch = (C + 7) / 8;
    if (C < 8) return {1, 1};
    for (int l : {8, 16, 32, 64})
        if (ch <= l) return {l, 1};
    if (ch <= 128) return backward ? Group{64, 2} : Group{128, 1};
    if (ch <= 256) return {256, 1};
    if (ch <= 512) return {256, 2};
    if (ch <= 1024) return {512, 2};
    return {0, 0};
}

template <bool BACKWARD, typename F>
hipError_t with_group(const Group &g, F f)
{
    using std::integral_constant;
#define IM2WIN_GROUP(L, K) \
    if (g.lpr == L && g.kch == K) return f(integral_constant<int, L>{}, integral_constant<int, K>{});
    IM2WIN_GROUP(1, 1)
    IM2WIN_GROUP(8, 1)
    IM2WIN_GROUP(16, 1)
    IM2WIN_GROUP(32, 1)
    IM2WIN_GROUP(64, 1)
    if constexpr (BACKWARD) {
        IM2WIN_GROUP(64, 2)
    } else {
        IM2WIN_GROUP(128, 1)
    }
    IM2WIN_GROUP(256, 1)
    IM2WIN_GROUP(256, 2)
    IM2WIN_GROUP(512, 2)
#undef IM2WIN_GROUP
    return hipErrorInvalidValue;
}

// Workgroups: forward 16 waves to a CU (one chunk of 256 lanes: 32, two chunks: 8; 65536
// rows of 2048, bf16: 231 and 226 us with 16 and 32; 32768 of 4096: 214, 222 and 234 with 8,
// 12 and 16); backward one workgroup to a CU, since each leaves sums (200000 rows of 512,
// bf16: 265 us with one or two; 4096 channels 329 and 344).
int64_t blocks_of(int64_t N, const Group &g, bool backward)
{
    const int64_t threads = threads_of(g.lpr), per = threads / g.lpr;
    const int64_t waves = g.kch > 1 ? 8 : g.lpr == 256 ? 32 : 16;
    const int64_t most = backward ? 256 : 256 * waves / (threads / 64);
    return std::max<int64_t>(1, std::min((N + per - 1) / per, most));
}
constexpr int64_t kWideBlocks = 2048, kColBlocks = 32;

int64_t bwd_blocks(int64_t N, int64_t C)
{
    const Group g = group_of(C, true);
    return g.lpr ? blocks_of(N, g, true) : std::max<int64_t>(1, std::min(N, kColBlocks));
}

// Whether each row's lanes take whole groups of rows with a gate: where groups are short,
// or where a workgroup would leave sums so often that this takes longer than the lanes wait
// which have no group, or the last ones. `share`: of the lanes' time that has a group in it.
// us of a workgroup's rows group by group, and so:
//   up to 256 channels (whose sums leave 8 rows' lanes after each other), from a quarter on:
//     65536 rows of 64, bf16, 65536 groups 2796 and 39, 2048 (a quarter) 111 and 53
//   up to 512, from three quarters on: 32768 rows of 512, 512 groups (half) 59 and 75
//   up to 1024, from half on: 16384 rows of 1024, 512 groups (half) 73 and 65, 384 68 and 77
//   up to 4096, from three quarters on: 16384 rows of 4096, 192 groups (three quarters) 214
//     and 186, 128 204 and 248; of 2048, 192 118 and 118, 160 119 and 137, 2048 254 and 106
//   up to 8192, where lanes that keep the gates' sums too have the fewest registers, with two
//     groups to each: 8192 rows of 8192, 1024 groups 481 and 388, 512 351 and 358, 256 288
//     and 342, 128 242 and 502; fp32, 512 715 and 541, 256 651 and 525
//   rows <= 8: 3000 of 512, fp32, 375 groups (a third) 31 and 24; 1024 of 8192, bf16, 128
//     groups 106 and 89, 512 rows of 64 groups 73 and 79
bool own_groups(int64_t N, int64_t groups, const Group &g)
{
    if (!g.lpr || groups <= 1) return false;
    if (N / groups <= 8) return true;
    const int64_t units = 256 * (threads_of(g.lpr) / g.lpr), rounds = (groups + units - 1) / units;
    if (g.lpr == 512) return groups >= 2 * units;
    const int64_t quarters = g.lpr < 64 ? 1 : g.lpr == 64 && g.kch == 2 ? 2 : 3;
    return 4 * groups >= quarters * units * rounds;
}

}  // namespace

int64_t res_norm_bwd_ws_bytes(int64_t N, int64_t C, int64_t groups)
{
    const Group g = group_of(C, true);
    // (lanes that take whole groups leave one record a workgroup)
    const int64_t B = bwd_blocks(N, C), G = own_groups(N, groups, g) ? 1 : std::max<int64_t>(groups, 1);
    return ((2 * B + G) * 2 * C * 4 + (B + G + 1) / 2 * 8 + (g.lpr ? 0 : N * 8) + 255) / 256 * 256;
}

hipError_t launch_res_norm_fwd(const ResNormArgs &a, hipStream_t s)
{
    const Group g = group_of(a.C, false);
    return with_norm_types(a.dtype, a.branch_dtype, [&](auto tr, auto tb) {
        using TR = typename decltype(tr)::type;
        using TB = typename decltype(tb)::type;
        if (!g.lpr) {
            hipLaunchKernelGGL((res_norm_fwd_wide_kernel<TR, TB>), dim3(unsigned(std::min(a.N, kWideBlocks))),
                               dim3(kThreads), 0, s, a);
            return hipGetLastError();
        }
        return with_group<false>(g, [&](auto lpr, auto kch) {
            constexpr int LPR = decltype(lpr)::value, KCH = decltype(kch)::value;
            const dim3 grid(unsigned(blocks_of(a.N, g, false))), threads(threads_of(LPR));
            if constexpr (LPR > 1)
                if (a.C % 8 == 0) {
                    hipLaunchKernelGGL((res_norm_fwd_kernel<TR, TB, LPR, KCH, true>), grid, threads, 0, s, a);
                    return hipGetLastError();
                }
            hipLaunchKernelGGL((res_norm_fwd_kernel<TR, TB, LPR, KCH, false>), grid, threads, 0, s, a);
            return hipGetLastError();
        });
    });
}

hipError_t launch_res_norm_bwd(const ResNormArgs &a, hipStream_t s)
{
    if (a.N == 0) {
        const int64_t n = std::max<int64_t>(a.groups, 1) * a.C;
        hipLaunchKernelGGL(res_norm_zero_kernel, dim3(unsigned(std::min<int64_t>((n + 255) / 256, 4096))),
                           dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    const Group g = group_of(a.C, true);
    const int64_t B = bwd_blocks(a.N, a.C);
    const bool own = own_groups(a.N, a.groups, g);
    const hipError_t e = with_norm_types(a.dtype, a.branch_dtype, [&](auto tr, auto tb) {
        using TR = typename decltype(tr)::type;
        using TB = typename decltype(tb)::type;
        if (!g.lpr) {
            hipLaunchKernelGGL((res_norm_bwd_wide_kernel<TR, TB>), dim3(unsigned(std::min(a.N, kWideBlocks))),
                               dim3(kThreads), 0, s, a, a.ws ? sums_of(a, B).means : nullptr);
            const hipError_t e1 = hipGetLastError();
            if (e1 != hipSuccess || !a.ws) return e1;
            hipLaunchKernelGGL((res_norm_cols_kernel<TR, TB>), dim3(unsigned((a.C + 511) / 512), unsigned(B)),
                               dim3(kThreads), 0, s, a);
            return hipGetLastError();
        }
        return with_group<true>(g, [&](auto lpr, auto kch) {
            constexpr int LPR = decltype(lpr)::value, KCH = decltype(kch)::value;
            const dim3 threads(threads_of(LPR));
            const auto launch = [&](auto exact) {
                constexpr bool EXACT = decltype(exact)::value;
                if (own)
                    hipLaunchKernelGGL((res_norm_bwd_kernel<TR, TB, LPR, KCH, EXACT, true>), dim3(unsigned(B)), threads, 0, s,
                                       a);
                else
                    hipLaunchKernelGGL((res_norm_bwd_kernel<TR, TB, LPR, KCH, EXACT, false>), dim3(unsigned(B)), threads, 0,
                                       s, a);
                return hipGetLastError();
            };
            if constexpr (LPR > 1)
                if (a.C % 8 == 0) return launch(std::true_type{});
            return launch(std::false_type{});
        });
    });
    if (e != hipSuccess || !a.ws) return e;
    ResNormArgs j = a;
    if (own) {                                 // dgate is there, dpw and dpb one sum per workgroup
        j.gate = nullptr;
        j.dgate = nullptr;
        j.groups = 0;
    }
    const int W = join_channels(a.C);
    const int64_t G = std::max<int64_t>(j.groups, 1), tiles = (a.C + W - 1) / W;
    const int64_t gates = !j.dgate ? 0 : short_groups(B, G) ? (G * a.C + 255) / 256 : G * tiles;
    hipLaunchKernelGGL(res_norm_join_kernel, dim3(unsigned(std::min<int64_t>(2 * tiles + gates, 8192))), dim3(1024), 0, s,
                       j, B);
    return hipGetLastError();
}

}  // namespace im2win
