// Gated feed-forward block (im2win_block.h): the plan, the small kernels, the kernels
// for few rows, and the sequence of launches.
//
// Forward: the gate launch (ff_tiles.hip) forms both projections, the activation and
// the product and leaves h; a plain product (ff_products.hip) leaves y. Backward: the
// back launch leaves da and du from dy, Wd and the saved a and u; then dx, dWd and
// dWg with dWu.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ff_common.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

// ---- rows padded to whole granules, the largest |dy| -------------------------------

struct PadJob {
    const void *src;
    void *dst;
    int64_t ld, rows, D, Dp; // elements; dst [rows][Dp]
    int64_t end;             // workgroups up to and with this job's
};
struct PadArgs {
    PadJob job[5];
    int count;
    const void *dy;          // of which the largest finite |value| is wanted, or null
    int64_t lddy, N, O;
    float *amax;             // [kAmaxParts]: of every kAmaxParts-th row
};

template <typename T>
__global__ __launch_bounds__(256) void ff_pad_kernel(const PadArgs a)
{
    constexpr int E = 16 / int(sizeof(T));
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t copies = a.count ? a.job[a.count - 1].end : 0;
    int64_t b = blockIdx.x;
    if (b >= copies) {
        __shared__ float red[4];
        b -= copies;
        float m = 0.f;
        for (int64_t r = b; r < a.N; r += kAmaxParts)
            for (int64_t c = threadIdx.x * E; c < a.O; c += 256 * E) {
                float f[E];
                load_some<E>(static_cast<const T *>(a.dy) + r * a.lddy + c, a.O - c, f);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (fabsf(f[e]) < __builtin_inff()) m = fmaxf(m, fabsf(f[e]));
            }
        for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
        if (lane == 0) red[wave] = m;
        __syncthreads();
        if (threadIdx.x == 0) a.amax[b] = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        return;
    }
    int k = 0;
    while (b >= a.job[k].end) ++k;
    const PadJob &j = a.job[k];
    const int64_t row = (b - (k ? a.job[k - 1].end : 0)) * 4 + wave;
    if (row >= j.rows) return;
    for (int64_t c = lane * E; c < j.Dp; c += 64 * E) {
        float f[E];
        load_some<E>(static_cast<const T *>(j.src) + row * j.ld + c, std::min<int64_t>(E, j.D - c), f);
        store_vec<E>(static_cast<T *>(j.dst) + row * j.Dp + c, f);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void ff_zero_kernel(T *p, int64_t n)
{
    const int64_t step = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) p[i] = T(0.f);
}

// ---- few rows ------------------------------------------------------------------------
//
// At most 16 rows: the weights are read once and that read is all that counts. A
// workgroup takes 16 rows of a weight matrix (of Wg and of Wu for h), its waves split
// K; the weights go from memory straight to the lanes that multiply them (16 rows x 64
// bytes a load, the matrix cores' own layout, so no LDS and no barrier until the waves'
// sums are joined), x or h come from the caches. Rows past N repeat the last one and
// are not stored.

// K values at `k` of a row of K: whole vectors in the steps below `whole`, else up to
// the row's end and zeros past it
template <typename T>
__device__ __forceinline__ uint4 row_frag(const T *row, int64_t k, int64_t K, bool whole)
{
    constexpr int E = 16 / int(sizeof(T));
    if (whole) {
        const Raw<T, E> r = load_raw<T, E>(row + k);
        return uint4{r.d[0], r.d[1], r.d[2], r.d[3]};
    }
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (k + e < K) {
            if constexpr (sizeof(T) == 4)
                d[e] = __float_as_uint(row[k + e]);
            else
                d[e / 2] |= uint32_t(__builtin_bit_cast(uint16_t, row[k + e])) << (e & 1) * 16;
        }
    return uint4{d[0], d[1], d[2], d[3]};
}

template <typename T>
constexpr int kFragK = 64 / int(sizeof(T));    // K of a fragment pair: 16 bytes a lane

// the waves' sums in order, left with the first wave
template <int WAVES, int NB>
__device__ __forceinline__ void join_parts(floatx4_t (&acc)[NB], floatx4_t *part)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave > 0)
#pragma unroll
        for (int i = 0; i < NB; ++i) part[((wave - 1) * NB + i) * 64 + lane] = acc[i];
    __syncthreads();
    if (wave > 0) return;
    for (int w = 1; w < WAVES; ++w)
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] += part[((w - 1) * NB + i) * 64 + lane];
}

template <typename T, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void ff_rows_gate_kernel(const FfRows a)
{
    constexpr int KF = kFragK<T>, U = 4;       // fragments in flight per matrix
    __shared__ floatx4_t part[(WAVES - 1) * 2 * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t f0 = int64_t(blockIdx.x) * 16, f = min(f0 + (lane & 15), a.F - 1);
    const int64_t n = min(int64_t(lane & 15), a.N - 1);
    const T *wg = static_cast<const T *>(a.wg) + f * a.ldg, *wu = static_cast<const T *>(a.wu) + f * a.ldu;
    const T *x = static_cast<const T *>(a.x) + n * a.ldx;
    const int q = (lane >> 4) * (16 / int(sizeof(T)));
    const int64_t steps = (a.D + KF - 1) / KF, whole = a.D / KF;
    int64_t s = steps * wave / WAVES;
    const int64_t end = steps * (wave + 1) / WAVES;
    floatx4_t acc[2] = {};
    for (; s + U <= min(end, whole); s += U) {
        uint4 g[U], u[U], b[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            g[i] = row_frag(wg, (s + i) * KF + q, a.D, true);
            u[i] = row_frag(wu, (s + i) * KF + q, a.D, true);
            b[i] = row_frag(x, (s + i) * KF + q, a.D, true);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            acc[0] = mfma_half<T>(g[i], b[i], acc[0]);
            acc[1] = mfma_half<T>(u[i], b[i], acc[1]);
        }
    }
    for (; s < end; ++s) {
        const uint4 b = row_frag(x, s * KF + q, a.D, s < whole);
        acc[0] = mfma_half<T>(row_frag(wg, s * KF + q, a.D, s < whole), b, acc[0]);
        acc[1] = mfma_half<T>(row_frag(wu, s * KF + q, a.D, s < whole), b, acc[1]);
    }
    join_parts<WAVES, 2>(acc, part);
    if (wave > 0 || (lane & 15) >= a.N) return;
    float h[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        float g, dg;
        activate<sizeof(T) == 4>(a.act, acc[0][v], g, dg);
        h[v] = g * acc[1][v];
    }
    const int64_t m = f0 + (lane >> 4) * 4;
    store_some<4>(a.h + (lane & 15) * a.F + m, a.F - m, h);
}

// y from the fp32 h: half precision as the sum of a rounded h and what that took
template <typename T, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void ff_rows_down_kernel(const FfRows a)
{
    constexpr int KF = kFragK<T>, E = 16 / int(sizeof(T)), U = 4;
    __shared__ floatx4_t part[(WAVES - 1) * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t o0 = int64_t(blockIdx.x) * 16, o = min(o0 + (lane & 15), a.O - 1);
    const int64_t n = min(int64_t(lane & 15), a.N - 1);
    const T *w = static_cast<const T *>(a.wd) + o * a.ldd;
    const float *h = a.h + n * a.F;
    const int q = (lane >> 4) * E;
    const int64_t steps = (a.F + KF - 1) / KF, whole = a.F / KF;
    int64_t s = steps * wave / WAVES;
    const int64_t end = steps * (wave + 1) / WAVES;
    floatx4_t acc[1] = {};
    auto multiply = [&](const uint4 &wf, const float (&f)[E]) {
        if constexpr (sizeof(T) == 4) {
            acc[0] = mfma_half<T>(wf, uint4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                            __float_as_uint(f[3])}, acc[0]);
        } else {
            const Raw<T, 8> hi = to_raw<T, 8>(f);
            float rest[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) rest[e] = f[e] - element(hi, e);
            const Raw<T, 8> lo = to_raw<T, 8>(rest);
            acc[0] = mfma_half<T>(wf, uint4{hi.d[0], hi.d[1], hi.d[2], hi.d[3]}, acc[0]);
            acc[0] = mfma_half<T>(wf, uint4{lo.d[0], lo.d[1], lo.d[2], lo.d[3]}, acc[0]);
        }
    };
    for (; s + U <= min(end, whole); s += U) {
        uint4 wf[U];
        float f[U][E];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            wf[i] = row_frag(w, (s + i) * KF + q, a.F, true);
            load_vec<E>(h + (s + i) * KF + q, f[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) multiply(wf[i], f[i]);
    }
    for (; s < end; ++s) {
        float f[E];
        load_some<E>(h + s * KF + q, max(int64_t(0), a.F - s * KF - q), f);
        multiply(row_frag(w, s * KF + q, a.F, s < whole), f);
    }
    join_parts<WAVES, 1>(acc, part);
    if (wave > 0 || (lane & 15) >= a.N) return;
    const int64_t m = o0 + (lane >> 4) * 4;
    const float y[4] = {acc[0][0], acc[0][1], acc[0][2], acc[0][3]};
    store_some<4>(static_cast<T *>(a.y) + (lane & 15) * a.ldy + m, a.O - m, y);
}

// ---- plan ------------------------------------------------------------------------------

struct FfPlan {
    bool few;                // the kernels for few rows
    int64_t Dp, Fp, Op, rows_pad, fblocks;
    bool copy_x, copy_g, copy_u, copy_d, copy_y;   // rows not made of 16-byte granules
    int gate_tile, y_tile, y_split, back_tile, dx_tile, dx_split, dd_tile, dd_split, dg_tile, dg_split;
    int64_t off_x, off_g, off_u, off_d, off_dy, off_h, off_slab_x, off_slab_d, off_slab_g, off_grad, off_amax, bytes;
    int64_t pre_bytes;       // of saved, before h
};

int64_t take(FfPlan &p, int64_t bytes)
{
    const int64_t at = p.bytes;
    p.bytes += round_up(bytes, 256);
    return at;
}

// tile of a product that is not split
int pick_tile(int64_t M, int64_t N, int64_t stages, int dtype, int out_bytes)
{
    double best = 1e30;
    int tile = 0;
    for (int t = 0; t < 3; ++t) {
        const double us = product_us(kShapes[t], M, N, stages, 1, dtype, out_bytes);
        if (us < best * 0.98) {
            best = us;
            tile = t;
        }
    }
    return tile;
}

FfPlan plan_common(const FfSizes &z)
{
    FfPlan p{};
    const int64_t es = elem(z.dtype), e = 16 / es;
    p.Dp = round_up(z.D, e);
    p.Fp = round_up(z.F, e);
    p.Op = round_up(z.O, e);
    p.rows_pad = round_up(z.N, 128 / es);
    // whole tiles: the back launch's reads need no bounds
    p.fblocks = round_up(z.F, 256) / 16;
    p.pre_bytes = round_up(z.N, 256) / 16 * p.fblocks * 2048;
    p.copy_x = z.D % e != 0 || z.ldx % e != 0;
    p.copy_g = z.D % e != 0 || z.ldg % e != 0;
    p.copy_u = z.D % e != 0 || z.ldu % e != 0;
    p.copy_d = z.F % e != 0 || z.ldd % e != 0;
    p.copy_y = z.O % e != 0 || z.ldy % e != 0;
    return p;
}

// what either pass reads as whole granules
void plan_copies(FfPlan &p, const FfSizes &z)
{
    const int64_t es = elem(z.dtype);
    if (p.copy_x) p.off_x = take(p, z.N * p.Dp * es);
    if (p.copy_g) p.off_g = take(p, z.F * p.Dp * es);
    if (p.copy_u) p.off_u = take(p, z.F * p.Dp * es);
    if (p.copy_d) p.off_d = take(p, z.O * p.Fp * es);
}

FfPlan plan_fwd(const FfSizes &z, bool saved)
{
    FfPlan p = plan_common(z);
    if (z.N == 0) return p;
    const int64_t es = elem(z.dtype), ki = 128 / es;
    p.few = z.N <= FF_ROWS && !saved;
    if (p.few) {
        p.off_h = take(p, z.N * z.F * 4);
        return p;
    }
    plan_copies(p, z);
    if (!saved) p.off_h = take(p, p.rows_pad * p.Fp * es);
    p.gate_tile = pick_tile(2 * p.Fp, z.N, ceil_div(p.Dp, ki), z.dtype, int(saved ? 4 + es / 2 : es / 2));
    pick_product(z.O, z.N, ceil_div(p.Fp, ki), z.dtype, 0, &p.y_tile, &p.y_split);
    if (p.y_split > 1) p.off_slab_x = take(p, p.y_split * z.N * z.O * 4);
    return p;
}

FfPlan plan_bwd(const FfSizes &z)
{
    FfPlan p = plan_common(z);
    if (z.N == 0) return p;
    const int64_t es = elem(z.dtype), ki = 128 / es;
    plan_copies(p, z);
    if (p.copy_y) p.off_dy = take(p, z.N * p.Op * es);
    p.off_grad = take(p, p.rows_pad * 2 * p.Fp * es);
    p.off_amax = take(p, kAmaxParts * 4);
    p.back_tile = pick_tile(p.Fp, z.N, ceil_div(z.O, ki), z.dtype, int(8 + 2 * es));
    pick_product(z.D, z.N, 2 * ceil_div(z.F, ki), z.dtype, 0, &p.dx_tile, &p.dx_split);
    pick_product(z.F, z.O, ceil_div(z.N, ki), z.dtype, 0, &p.dd_tile, &p.dd_split);
    pick_product(z.D, 2 * z.F, ceil_div(z.N, ki), z.dtype, 0, &p.dg_tile, &p.dg_split);
    if (p.dx_split > 1) p.off_slab_x = take(p, p.dx_split * z.N * z.D * 4);
    if (p.dd_split > 1) p.off_slab_d = take(p, p.dd_split * z.O * z.F * 4);
    if (p.dg_split > 1) p.off_slab_g = take(p, p.dg_split * 2 * z.F * z.D * 4);
    return p;
}

// x, the weights and dy as rows of whole granules
struct FfRead {
    const void *x, *wg, *wu, *wd, *dy;
    int64_t ldx, ldg, ldu, ldd, lddy;          // bytes
};

hipError_t launch_pads(const FfPlan &p, const FfArgs &a, bool backward, FfRead *r, hipStream_t s)
{
    const FfSizes &z = a.z;
    const int64_t es = elem(z.dtype);
    char *ws = static_cast<char *>(a.ws);
    PadArgs pad{};
    int64_t groups = 0;
    auto add = [&](bool copy, const void *src, int64_t ld, int64_t rows, int64_t D, int64_t Dp, int64_t off,
                   const void *&to, int64_t &to_ld) {
        to = src;
        to_ld = ld * es;
        if (!copy) return;
        to = ws + off;
        to_ld = Dp * es;
        groups += ceil_div(rows, 4);
        pad.job[pad.count++] = PadJob{src, ws + off, ld, rows, D, Dp, groups};
    };
    add(p.copy_x, a.x, z.ldx, z.N, z.D, p.Dp, p.off_x, r->x, r->ldx);
    add(p.copy_g, a.wg, z.ldg, z.F, z.D, p.Dp, p.off_g, r->wg, r->ldg);
    add(p.copy_u, a.wu, z.ldu, z.F, z.D, p.Dp, p.off_u, r->wu, r->ldu);
    add(p.copy_d, a.wd, z.ldd, z.O, z.F, p.Fp, p.off_d, r->wd, r->ldd);
    if (backward) {
        add(p.copy_y, a.dy, z.ldy, z.N, z.O, p.Op, p.off_dy, r->dy, r->lddy);
        if (z.dtype == 1) {
            pad.dy = a.dy;
            pad.lddy = z.ldy;
            pad.N = z.N;
            pad.O = z.O;
            pad.amax = reinterpret_cast<float *>(ws + p.off_amax);
            groups += kAmaxParts;
        }
    }
    if (groups == 0) return hipSuccess;
    return with_ff_type(z.dtype, [&](auto t) {
        hipLaunchKernelGGL((ff_pad_kernel<decltype(t)>), dim3(unsigned(groups)), dim3(256), 0, s, pad);
        return hipGetLastError();
    });
}

FfSaved saved_of(const FfPlan &p, const void *saved, void *h)
{
    char *c = static_cast<char *>(const_cast<void *>(saved));
    return FfSaved{reinterpret_cast<float *>(c), p.fblocks, c ? c + p.pre_bytes : h};
}

// the waves of a workgroup that split K: a wave should have some steps of its own
template <typename T>
hipError_t launch_rows(const FfRows &a, hipStream_t s)
{
    const dim3 gate(unsigned(ceil_div(a.F, 16))), down(unsigned(ceil_div(a.O, 16)));
    hipLaunchKernelGGL((ff_rows_gate_kernel<T, 4>), gate, dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ff_rows_down_kernel<T, 16>), down, dim3(1024), 0, s, a);
    return hipGetLastError();
}

}  // namespace

int64_t ff_saved_bytes(const FfSizes &z)
{
    const FfPlan p = plan_common(z);
    return p.pre_bytes + p.rows_pad * p.Fp * elem(z.dtype);
}

int64_t ff_fwd_ws_bytes(const FfSizes &z, bool saved) { return plan_fwd(z, saved).bytes; }
int64_t ff_bwd_ws_bytes(const FfSizes &z) { return plan_bwd(z).bytes; }

hipError_t launch_ff_rows(const FfRows &a, int dtype, hipStream_t s)
{
    return with_ff_type(dtype, [&](auto t) { return launch_rows<decltype(t)>(a, s); });
}

hipError_t launch_ff_fwd(const FfArgs &a, hipStream_t s)
{
    const FfSizes &z = a.z;
    if (z.N == 0) return hipSuccess;
    const FfPlan p = plan_fwd(z, a.saved != nullptr);
    char *ws = static_cast<char *>(a.ws);
    const int64_t es = elem(z.dtype);
    if (p.few)
        return launch_ff_rows(FfRows{a.x, a.wg, a.wu, a.wd, z.ldx, z.ldg, z.ldu, z.ldd, z.ldy, z.N, z.D, z.F, z.O,
                                     reinterpret_cast<float *>(ws + p.off_h), a.y, z.act}, z.dtype, s);
    FfRead r{};
    hipError_t e = launch_pads(p, a, false, &r, s);
    if (e != hipSuccess) return e;
    const FfSaved to = saved_of(p, a.saved, ws + p.off_h);
    const FfGate g{r.x, r.wg, r.wu, r.ldx, r.ldg, r.ldu, z.N, z.F, p.Dp, p.rows_pad, p.Fp, to, z.act};
    if ((e = launch_ff_gate(g, z.dtype, p.gate_tile, s)) != hipSuccess) return e;
    FfProduct y{};
    y.a[0] = r.wd;
    y.lda[0] = r.ldd;
    y.b = to.h;
    y.ldb = p.Fp * es;
    y.M = y.a_count = z.O;
    y.n = y.b_count = z.N;
    y.K = y.k_a = y.k_b = p.Fp;
    y.segs = y.outs = 1;
    y.split = p.y_split;
    y.slab = p.y_split > 1 ? reinterpret_cast<float *>(ws + p.off_slab_x) : nullptr;
    y.out[0] = a.y;
    y.ldo = z.ldy;
    if ((e = launch_ff_y(y, z.dtype, p.y_tile, s)) != hipSuccess) return e;
    return y.slab ? launch_ff_join(&y, 1, z.dtype, s) : hipSuccess;
}

hipError_t launch_ff_bwd(const FfArgs &a, hipStream_t s)
{
    const FfSizes &z = a.z;
    const int64_t es = elem(z.dtype);
    if (z.N == 0)
        return with_ff_type(z.dtype, [&](auto t) {
            using T = decltype(t);
            const auto zero = [&](void *p, int64_t n) {
                const int64_t groups = std::min(ceil_div(n, 256), max_groups(256));
                hipLaunchKernelGGL((ff_zero_kernel<T>), dim3(unsigned(groups)), dim3(256), 0, s, static_cast<T *>(p), n);
            };
            zero(a.dwg, z.F * z.D);
            zero(a.dwu, z.F * z.D);
            zero(a.dwd, z.O * z.F);
            return hipGetLastError();
        });
    const FfPlan p = plan_bwd(z);
    char *ws = static_cast<char *>(a.ws);
    FfRead r{};
    hipError_t e = launch_pads(p, a, true, &r, s);
    if (e != hipSuccess) return e;
    const float *amax = z.dtype == 1 ? reinterpret_cast<const float *>(ws + p.off_amax) : nullptr;
    const FfSaved from = saved_of(p, a.saved, nullptr);
    const FfBack back{r.dy, r.wd, r.lddy, r.ldd, z.N, z.F, z.O, p.Op, p.rows_pad, p.Fp, from, ws + p.off_grad, amax, z.act};
    if ((e = launch_ff_back(back, z.dtype, p.back_tile, s)) != hipSuccess) return e;

    FfProduct dx{}, dd{}, dg{};
    dx.a[0] = r.wg;
    dx.a[1] = r.wu;
    dx.lda[0] = r.ldg;
    dx.lda[1] = r.ldu;
    dx.b = dg.b = ws + p.off_grad;
    dx.b_step = dg.b_step = p.Fp * es;
    dx.ldb = dg.ldb = 2 * p.Fp * es;
    dx.M = dg.M = z.D;
    dx.a_count = dg.a_count = p.Dp;
    dx.n = dx.b_count = z.N;
    dx.K = dx.k_a = z.F;
    dx.k_b = p.Fp;
    dx.segs = 2;
    dx.outs = 1;
    dx.split = p.dx_split;
    dx.slab = p.dx_split > 1 ? reinterpret_cast<float *>(ws + p.off_slab_x) : nullptr;
    dx.out[0] = a.dx;
    dx.ldo = dg.ldo = z.D;
    dx.amax = dg.amax = amax;

    dg.a[0] = r.x;
    dg.lda[0] = r.ldx;
    dg.n = z.F;
    dg.b_count = p.Fp;
    dg.K = dg.k_a = z.N;
    dg.k_b = p.rows_pad;
    dg.segs = 1;
    dg.outs = 2;
    dg.split = p.dg_split;
    dg.slab = p.dg_split > 1 ? reinterpret_cast<float *>(ws + p.off_slab_g) : nullptr;
    dg.out[0] = a.dwg;
    dg.out[1] = a.dwu;

    dd.a[0] = from.h;
    dd.lda[0] = p.Fp * es;
    dd.b = r.dy;
    dd.ldb = r.lddy;
    dd.M = z.F;
    dd.a_count = p.Fp;
    dd.n = z.O;
    dd.b_count = p.Op;
    dd.K = dd.k_b = z.N;
    dd.k_a = p.rows_pad;
    dd.segs = dd.outs = 1;
    dd.split = p.dd_split;
    dd.slab = p.dd_split > 1 ? reinterpret_cast<float *>(ws + p.off_slab_d) : nullptr;
    dd.out[0] = a.dwd;
    dd.ldo = z.F;

    if (p.dx_tile == kTile64 && p.dd_tile == kTile64 && p.dg_tile == kTile64) {
        if ((e = launch_ff_all(dx, dd, dg, z.dtype, s)) != hipSuccess) return e;
    } else {
        if ((e = launch_ff_dx(dx, z.dtype, p.dx_tile, s)) != hipSuccess) return e;
        if ((e = launch_ff_dw(dd, z.dtype, p.dd_tile, s)) != hipSuccess) return e;
        if ((e = launch_ff_dw(dg, z.dtype, p.dg_tile, s)) != hipSuccess) return e;
    }
    FfProduct join[3];
    int count = 0;
    for (const FfProduct *q : {&dx, &dd, &dg})
        if (q->slab) join[count++] = *q;
    return count ? launch_ff_join(join, count, z.dtype, s) : hipSuccess;
}

}  // namespace im2win
