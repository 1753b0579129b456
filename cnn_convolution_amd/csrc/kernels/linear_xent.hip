// Softmax cross entropy of a linear classifier (im2win_head.h): the plan, the
// small kernels, and the sequence of launches.
//
// Forward: one launch of logit tiles (xent_logits.hip) leaves each row's
// (maximum, sum of exponentials) per tile of classes, a second joins them.
// Backward, in pieces of the classes: a piece's G goes to the workspace
// (xent_logits.hip), then dx += G w and dw = G^T x (xent_products.hip).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>

#include "../xent.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

__device__ __forceinline__ bool valid_target(int64_t t, int64_t V) { return t >= 0 && t < V; }

// (m, s) joined by (m2, s2). A part without a class, or of classes at -infinity
// alone, is (-infinity, 0) and adds nothing. NaN is in a part's sum only: fmaxf passes
// it over, and a tile of NaN classes and padding has the maximum -infinity, so it is
// by the sum that a part is left out (as a choice, not a branch: the next part's load
// would be waited for behind it).
__device__ __forceinline__ void join_part(float &m, float &s, float m2, float s2)
{
    const float n = fmaxf(m, m2), a = s * __expf(m - n), b = s2 * __expf(m2 - n);
    s = (s == 0.f ? 0.f : a) + (s2 == 0.f ? 0.f : b);
    m = n;
}

// one wave per row: lse over the tiles' partials, then the loss
__global__ __launch_bounds__(256) void xent_join_kernel(const XentArgs a, const float2 *partial, int tiles)
{
    const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= a.N) return;
    float m = -__builtin_inff(), s = 0.f;
    for (int t = lane; t < tiles; t += 64) {
        const float2 p = partial[t * a.N + row];
        join_part(m, s, p.x, p.y);
    }
    for (int k = 1; k < 64; k <<= 1) {
        const float m2 = __shfl_xor(m, k, 64), s2 = __shfl_xor(s, k, 64);
        join_part(m, s, m2, s2);
    }
    if (lane == 0) {
        const float lse = m + logf(s);
        const bool ok = valid_target(a.target[row], a.V);
        // a small loss of large logits: the maximum cancels before the rounding of lse
        a.loss[row] = ok ? logf(s) + (m - a.loss[row]) : 0.f;
        a.lse[row] = ok ? lse : 0.f;
    }
}

// S: the power of two with S * max |grad| in [2^14, 2^15], by one workgroup. The
// maximum is over the rows that have a gradient: a masked row's grad may hold
// anything, and an infinite (or NaN) one is its own row's affair.
template <int THREADS>
__device__ __forceinline__ void grad_scale(const float *grad, const int64_t *target, int64_t V, int64_t N,
                                           float *scale)
{
    __shared__ float red[THREADS / 64];
    float m = 0.f;
    for (int64_t i = threadIdx.x; i < N; i += THREADS) {
        const float g = fabsf(grad[i]);
        if (valid_target(target[i], V) && g < __builtin_inff()) m = fmaxf(m, g);
    }
    for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < THREADS / 64; ++w) m = fmaxf(m, red[w]);
        int e = 0;
        const bool ok = m > 0.f;
        if (ok) (void)frexpf(m, &e);
        e = max(-100, min(100, 15 - e));
        scale[0] = ok ? ldexpf(1.f, e) : 1.f;
        scale[1] = ok ? ldexpf(1.f, -e) : 1.f;
    }
}

__global__ __launch_bounds__(1024) void xent_scale_kernel(const float *grad, const int64_t *target, int64_t V,
                                                         int64_t N, float *scale)
{
    grad_scale<1024>(grad, target, V, N, scale);
}

// What the class weights share: per feature their mean where all have one sign, else 0,
// over up to 64 classes spread over all (dx takes no more of it than the weight of a
// row's own target). 256 features per workgroup, every fourth class a wave; beside the
// row copy, for whose launch it costs 0.8 us (64 rows, 1000 classes, 512 features, bf16:
// step 23.3 -> 24.8 us).
constexpr int kSharedRows = 64;
template <typename T>
__device__ __forceinline__ void shared_weights(const T *w, int64_t ldw, int64_t V, int64_t D, int64_t d0, float *shared,
                                               int *some)
{
    __shared__ float part[3][4][256];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t d = d0 + lane * 4;
    const int S = int(min(V, int64_t(kSharedRows)));
    const auto row = [&](int k) { return w + (S < V ? int64_t(k) * V / kSharedRows : k) * ldw; };
    float lo[4], hi[4], sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        lo[e] = __builtin_inff();
        hi[e] = -__builtin_inff();
        sum[e] = 0.f;
    }
    if (D >= 4) {
        // without branches: zeros past the row's end, the last class again past S
#pragma unroll
        for (int i = 0; i < kSharedRows / 4; ++i) {
            const Raw<T, 4> r = load_row<T, 4, false>(row(min(i * 4 + wave, S - 1)), d, D);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[e] = fminf(lo[e], element(r, e));
                hi[e] = fmaxf(hi[e], element(r, e));
                sum[e] += i * 4 + wave < S ? element(r, e) : 0.f;
            }
        }
    } else {
        for (int k = wave; k < S; k += 4) {
            float f[4];
            load_some<4>(row(k) + d, D - d, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[e] = fminf(lo[e], f[e]);
                hi[e] = fmaxf(hi[e], f[e]);
                sum[e] += f[e];
            }
        }
    }
    store_vec<4>(&part[0][wave][lane * 4], lo);
    store_vec<4>(&part[1][wave][lane * 4], hi);
    store_vec<4>(&part[2][wave][lane * 4], sum);
    __syncthreads();
    const int t = threadIdx.x;
    const float l = fminf(fminf(part[0][0][t], part[0][1][t]), fminf(part[0][2][t], part[0][3][t]));
    const float h = fmaxf(fmaxf(part[1][0][t], part[1][1][t]), fmaxf(part[1][2][t], part[1][3][t]));
    const float c = l > 0.f || h < 0.f
                        ? ((part[2][0][t] + part[2][1][t]) + (part[2][2][t] + part[2][3][t])) / float(S)
                        : 0.f;
    shared[d0 + t] = c;
    const int any = __syncthreads_or(c != 0.f);
    if (t == 0) some[d0 / 256] = any;
}

// rows copied to whole granules (the padding cleared), one wave per row; with
// targets also t32 (rows up to rows_pad), and masked rows copied as zeros. Further
// workgroups find the gradients' scale (one, with grad) and what the class weights
// share (one for each 256 features, with shared).
template <typename T>
__global__ __launch_bounds__(256) void xent_rows_kernel(const T *src, int64_t ld, int64_t rows, int64_t D, int64_t Dp,
                                                        T *dst, const int64_t *target, int64_t V, int64_t rows_pad,
                                                        int *t32, const float *grad, float *scale, const T *w,
                                                        int64_t ldw, float *shared, int *some)
{
    if (target && blockIdx.x >= rows_pad / 4) {
        const int64_t extra = blockIdx.x - rows_pad / 4;
        if (grad && extra == 0)
            grad_scale<256>(grad, target, V, rows, scale);
        else
            shared_weights(w, ldw, V, D, (extra - (grad ? 1 : 0)) * 256, shared, some);
        return;
    }
    const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    constexpr int E = 16 / int(sizeof(T));
    bool ok = row < rows;
    if (target) {
        const int64_t t = ok ? target[row] : -1;
        ok = valid_target(t, V);
        if (lane == 0 && row < rows_pad) t32[row] = ok ? int(t) : -1;
    }
    if (row >= rows) return;
    for (int64_t d = lane * E; d < Dp; d += 64 * E) {
        float f[E];
        load_some<E>(src + row * ld + d, ok ? int(min(int64_t(E), D - d)) : 0, f);
        store_vec<E>(dst + row * Dp + d, f);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void xent_zero_kernel(T *p, int64_t n)
{
    const int64_t step = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) p[i] = T(0.f);
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }
int64_t elem(int dtype) { return dtype == 0 ? 4 : 2; }

template <typename F>
hipError_t with_type(int dtype, F f)
{
    if (dtype == 0) return f(float{});
    if (dtype == 1) return f(_Float16{});
    return f(__bf16{});
}

// Time of one launch, from measurements of each tile shape (bf16 and fp32,
// 8192 x 16384 outputs over K 512 .. 4096, and single workgroups over K 8192):
// microseconds of a K stage with 1, 2, .. workgroups on a CU, and what a
// workgroup adds per tile. Half precision at K = 512, 1024, 4096 (TFLOP/s):
// 256 x 256 1079, 1168, 1418; 128 x 128 881, 984, 1163; 64 x 64 576, 669, 725;
// a lone 64 x 64 workgroup takes 0.30 us a stage, 128 x 128 0.69, 256 x 256 1.28.
struct Tile {
    int64_t m, n;
    int per_cu;              // workgroups a CU holds
    double half[4], f32[4];  // us per stage with 1, 2, .. of them
    double fixed;            // us per tile before its epilogue
};
constexpr Tile kShapes[5] = {{256, 256, 1, {1.42}, {7.3}, 4.3},
                             {128, 128, 2, {0.69, 0.88}, {1.9, 3.7}, 2.7},
                             {64, 64, 3, {0.30, 0.42, 0.53}, {0.48, 0.93, 1.4}, 1.3},
                             {32, 32, 1, {0.28}, {0.60}, 2.5},              // K over four waves
                             {64, 32, 4, {0.25, 0.30, 0.36, 0.42}, {0.30, 0.50, 0.73, 0.95}, 1.3}};
constexpr int64_t kCus = 256;

// microseconds of a product of M x N outputs over `stages` K stages that leaves
// out_bytes per output
double product_us(const Tile &t, int64_t M, int64_t N, int64_t stages, int split, int dtype, int out_bytes,
                  double hit_us = 0.0)
{
    const int64_t wgs = ceil_div(M, t.m) * ceil_div(N, t.n) * split;
    const int64_t of_cu = ceil_div(wgs, kCus);                    // the busiest CU's
    const auto held_us = [&](int64_t held) {
        if (held == 0) return 0.0;
        const double stage = (dtype == 0 ? t.f32 : t.half)[held - 1] + hit_us;
        // an epilogue: 7 us for 65536 exponentials on a CU, or its stores at a CU's
        // share of the memory bandwidth; half of it hidden by a neighbour's products
        const double outputs = double(held * t.m * t.n);
        const double epilogue = std::max(outputs * 7.0 / 65536, outputs * out_bytes / 2e4) * (held > 1 ? 0.5 : 1.0);
        return stage * double(ceil_div(stages, split)) + t.fixed + epilogue;
    };
    return double(of_cu / t.per_cu) * held_us(t.per_cu) + held_us(of_cu % t.per_cu);
}

constexpr int64_t kSlabBytes = int64_t(256) << 20;

// tile and split of a product whose K may be split
void pick_product(int64_t M, int64_t N, int64_t stages, int dtype, int64_t classes, int *tile, int *split)
{
    double best = 1e30;
    for (int t = 0; t < 3; ++t) {
        // dw in half precision: a stage of 64 rows with a target among a wave's 64
        // (tiles of 64: 32) classes takes about 0.9 us more
        const double hits = classes && dtype ? std::min(1.0, 64.0 * (kShapes[t].n == 64 ? 32 : 64) / double(classes)) : 0.0;
        for (int sp = 1; sp <= 64; sp *= 2) {
            if (sp > 1 && (stages / sp < 4 || int64_t(sp) * M * N * 4 > kSlabBytes)) break;
            // the slabs are read once more, at about 3 TB/s, by a launch of their own
            const double us = product_us(kShapes[t], M, N, stages, sp, dtype, sp > 1 ? 4 : int(elem(dtype)), 0.9 * hits) +
                              (sp > 1 ? 5.0 + double(sp) * double(M) * double(N) * 4 / 3e6 : 0.0);
            if (us < best * 0.98) {
                best = us;
                *tile = t;
                *split = sp;
            }
        }
    }
}

int pick_logits(int64_t M, int64_t N, int64_t stages, int dtype, bool narrow)
{
    if (narrow && N <= 16) return kTileNarrow;
    double best = 1e30;
    int tile = 0;
    for (int t = 0; t < 5; ++t) {
        const int64_t own = t == kTile32K ? ceil_div(stages, 4) : stages;
        const double us = product_us(kShapes[t], M, N, own, 1, dtype, narrow ? 0 : int(elem(dtype)));
        if (us < best * 0.98) {
            best = us;
            tile = t;
        }
    }
    return tile;
}

// Of G, but never less than 256 classes: with more than 2^18 rows (2^19 in half
// precision) a piece is those 256, 4 GB at 2^22 rows of fp32.
constexpr int64_t kPieceBytes = int64_t(256) << 20;

void plan_common(XentPlan &p, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    const int64_t e = 16 / elem(dtype);
    p.Dp = round_up(D, e);
    p.copy_x = D % e != 0 || ldx % e != 0;
    p.copy_w = D % e != 0 || ldw % e != 0;
}

int64_t take(XentPlan &p, int64_t bytes)
{
    const int64_t at = p.bytes;
    p.bytes += round_up(bytes, 256);
    return at;
}

}  // namespace

XentPlan plan_xent_fwd(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    XentPlan p{};
    plan_common(p, D, ldx, ldw, dtype);
    if (N == 0) return p;
    const int64_t es = elem(dtype);
    p.logits_tile = pick_logits(V, N, ceil_div(p.Dp * es, 128), dtype, true);
    p.tiles_v = ceil_div(V, p.logits_tile == kTileNarrow ? 128 : kShapes[p.logits_tile].m);
    if (p.copy_x) p.off_x = take(p, N * p.Dp * es);
    if (p.copy_w) p.off_w = take(p, V * p.Dp * es);
    p.off_partial = take(p, p.tiles_v * N * 8);
    return p;
}

XentPlan plan_xent_bwd(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    XentPlan p{};
    plan_common(p, D, ldx, ldw, dtype);
    p.copy_x = true;                      // the masked rows are cleared in it
    if (N == 0) return p;
    const int64_t es = elem(dtype), ki = 128 / es;
    p.rows_pad = round_up(N, 256);
    const int64_t most = std::max<int64_t>(1, kPieceBytes / (p.rows_pad * es) / 256) * 256;
    p.piece = std::min(round_up(V, 256), most);
    const int64_t P = std::min(V, p.piece);
    p.logits_tile = pick_logits(P, N, ceil_div(p.Dp * es, 128), dtype, false);
    pick_product(D, N, ceil_div(P, ki), dtype, 0, &p.dx_tile, &p.dx_split);
    pick_product(D, P, ceil_div(N, ki), dtype, V, &p.dw_tile, &p.dw_split);
    p.dx_direct = p.dx_split == 1 && P == V;
    p.off_scale = take(p, 8);
    p.off_t32 = take(p, p.rows_pad * 4);
    p.off_low = take(p, p.rows_pad * es);
    p.off_hits = take(p, p.piece / 32 * (p.rows_pad / 32));
    if (dtype) {
        p.off_rest = take(p, rest_blocks(p.logits_tile, P) * p.rows_pad * 4);
        p.off_shared = take(p, round_up(D, 256) * 4);
        p.off_some = take(p, round_up(D, 256) / 256 * 4);
    }
    p.off_x = take(p, N * p.Dp * es);
    if (p.copy_w) p.off_w = take(p, V * p.Dp * es);
    p.off_g = take(p, p.rows_pad * p.piece * es);
    if (!p.dx_direct) p.off_dx = take(p, p.dx_split * N * D * 4);
    if (p.dw_split > 1) p.off_dw = take(p, p.dw_split * P * D * 4);
    return p;
}

int64_t xent_fwd_ws_bytes(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    return plan_xent_fwd(N, V, D, ldx, ldw, dtype).bytes;
}

int64_t xent_bwd_ws_bytes(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype)
{
    return plan_xent_bwd(N, V, D, ldx, ldw, dtype).bytes;
}

hipError_t launch_xent_fwd(const XentArgs &a, hipStream_t s)
{
    if (a.N == 0) return hipSuccess;
    const XentPlan p = plan_xent_fwd(a.N, a.V, a.D, a.ldx, a.ldw, a.dtype);
    char *ws = static_cast<char *>(a.ws);
    const int64_t es = elem(a.dtype);
    LossArgs l{};
    l.r = XentRows{a.x, a.w, a.ldx * es, a.ldw * es};
    const hipError_t e = with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        if (p.copy_x) {
            l.r.x = ws + p.off_x;
            l.r.ldx = p.Dp * es;
            hipLaunchKernelGGL((xent_rows_kernel<T>), dim3(unsigned(ceil_div(a.N, 4))), dim3(256), 0, s,
                               static_cast<const T *>(a.x), a.ldx, a.N, a.D, p.Dp,
                               reinterpret_cast<T *>(ws + p.off_x), nullptr, a.V, 0, nullptr, nullptr,
                               nullptr, nullptr, 0, nullptr, nullptr);
        }
        if (p.copy_w) {
            l.r.w = ws + p.off_w;
            l.r.ldw = p.Dp * es;
            hipLaunchKernelGGL((xent_rows_kernel<T>), dim3(unsigned(ceil_div(a.V, 4))), dim3(256), 0, s,
                               static_cast<const T *>(a.w), a.ldw, a.V, a.D, p.Dp,
                               reinterpret_cast<T *>(ws + p.off_w), nullptr, a.V, 0, nullptr, nullptr,
                               nullptr, nullptr, 0, nullptr, nullptr);
        }
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    l.N = a.N;
    l.V = a.V;
    l.Dp = p.Dp;
    l.target = a.target;
    l.loss = a.loss;
    l.partial = reinterpret_cast<float2 *>(ws + p.off_partial);
    const hipError_t e2 = launch_xent_loss(l, a.dtype, p.logits_tile, s);
    if (e2 != hipSuccess) return e2;
    hipLaunchKernelGGL(xent_join_kernel, dim3(unsigned(ceil_div(a.N, 4))), dim3(256), 0, s, a, l.partial,
                       int(p.tiles_v));
    return hipGetLastError();
}

hipError_t launch_xent_bwd(const XentArgs &a, hipStream_t s)
{
    const XentPlan p = plan_xent_bwd(a.N, a.V, a.D, a.ldx, a.ldw, a.dtype);
    char *ws = static_cast<char *>(a.ws);
    const int64_t es = elem(a.dtype), ki = 128 / es;
    if (a.N == 0)
        return with_type(a.dtype, [&](auto t) {
            using T = decltype(t);
            const int64_t n = a.V * a.D;
            const int64_t groups = std::min(ceil_div(n, 256), max_groups(256));
            hipLaunchKernelGGL((xent_zero_kernel<T>), dim3(unsigned(groups)), dim3(256), 0, s, static_cast<T *>(a.dw),
                               n);
            return hipGetLastError();
        });
    float *scale = a.dtype == 1 ? reinterpret_cast<float *>(ws + p.off_scale) : nullptr;
    float *shared = a.dtype ? reinterpret_cast<float *>(ws + p.off_shared) : nullptr;
    int *some = a.dtype ? reinterpret_cast<int *>(ws + p.off_some) : nullptr;
    float *rest = a.dtype ? reinterpret_cast<float *>(ws + p.off_rest) : nullptr;
    int *t32 = reinterpret_cast<int *>(ws + p.off_t32);
    XentRows r{ws + p.off_x, a.w, p.Dp * es, a.ldw * es};
    hipError_t e = with_type(a.dtype, [&](auto t) {
        using T = decltype(t);
        // a workgroup of the copy has time for some tens of thousands of gradients
        const bool with_rows = scale && a.N <= 32768;
        if (scale && !with_rows)
            hipLaunchKernelGGL(xent_scale_kernel, dim3(1), dim3(1024), 0, s, a.grad, a.target, a.V, a.N, scale);
        const int64_t groups = p.rows_pad / 4 + (with_rows ? 1 : 0) + (shared ? round_up(a.D, 256) / 256 : 0);
        hipLaunchKernelGGL((xent_rows_kernel<T>), dim3(unsigned(groups)), dim3(256), 0, s,
                           static_cast<const T *>(a.x), a.ldx, a.N, a.D, p.Dp, reinterpret_cast<T *>(ws + p.off_x),
                           a.target, a.V, p.rows_pad, t32, with_rows ? a.grad : nullptr, scale,
                           static_cast<const T *>(a.w), a.ldw, shared, some);
        if (p.copy_w) {
            r.w = ws + p.off_w;
            r.ldw = p.Dp * es;
            hipLaunchKernelGGL((xent_rows_kernel<T>), dim3(unsigned(ceil_div(a.V, 4))), dim3(256), 0, s,
                               static_cast<const T *>(a.w), a.ldw, a.V, a.D, p.Dp,
                               reinterpret_cast<T *>(ws + p.off_w), nullptr, a.V, 0, nullptr, nullptr,
                               nullptr, nullptr, 0, nullptr, nullptr);
        }
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;

    ProductArgs dx{}, dw{};
    dx.t32 = dw.t32 = t32;
    dx.low = dw.low = ws + p.off_low;
    dw.hits = reinterpret_cast<uint8_t *>(ws + p.off_hits);
    dw.ldh = p.rows_pad / 32;
    dx.scale = dw.scale = scale;
    dx.b = dw.b = ws + p.off_g;
    dx.ldb = dw.ldb = p.piece * es;
    dx.M = dw.M = a.D;
    dx.lda = r.ldw;
    dx.w = r.w;
    dx.ldw = r.ldw;
    dx.n = a.N;
    dx.split = p.dx_split;
    dx.slab = p.dx_direct ? nullptr : reinterpret_cast<float *>(ws + p.off_dx);
    dx.out = a.dx;
    dx.rest = rest;
    dx.ldr = p.rows_pad;
    dx.shared = shared;
    dw.a = r.x;
    dw.lda = r.ldx;
    dw.K = dw.k_a = a.N;
    dw.k_b = p.rows_pad;
    dw.split = p.dw_split;
    dw.slab = p.dw_split > 1 ? reinterpret_cast<float *>(ws + p.off_dw) : nullptr;
    for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
        const int64_t P = std::min(p.piece, a.V - v0);
        GradArgs g{r, a.N, v0, P, p.Dp, t32, a.grad, a.lse, scale, ws + p.off_g, p.piece, ws + p.off_low,
                   reinterpret_cast<uint8_t *>(ws + p.off_hits), p.rows_pad / 32, rest, p.rows_pad,
                   some, int(ceil_div(a.D, 256))};
        if ((e = launch_xent_g(g, a.dtype, p.logits_tile, s)) != hipSuccess) return e;
        dx.a = static_cast<const char *>(r.w) + v0 * r.ldw;
        dx.K = dx.k_a = P;
        dx.k_b = round_up(P, ki);
        dx.blocks = int(rest_blocks(p.logits_tile, P));
        dx.add = v0 > 0;
        // a last piece of few stages: no part without one
        dx.split = int(std::min<int64_t>(p.dx_split, ceil_div(P, ki)));
        dw.n = P;
        dw.v0 = v0;
        dw.out = static_cast<char *>(a.dw) + v0 * a.D * es;
        if (p.dx_tile == kTile64 && p.dw_tile == kTile64) {
            if ((e = launch_xent_both(dx, dw, a.dtype, s)) != hipSuccess) return e;
        } else {
            if ((e = launch_xent_dx(dx, a.dtype, p.dx_tile, s)) != hipSuccess) return e;
            if ((e = launch_xent_dw(dw, a.dtype, p.dw_tile, s)) != hipSuccess) return e;
        }
        const bool done = v0 + P == a.V;
        dx.split = p.dx_split;
        if (dw.slab || (done && dx.slab)) {
            e = launch_xent_join(done && dx.slab ? &dx : nullptr, dw.slab ? &dw : nullptr, a.dtype, s);
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace im2win
