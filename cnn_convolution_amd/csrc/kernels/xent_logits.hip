// Logit tiles of the linear cross entropy: l[n][v] = sum_d w[v][d] x[n][d], with
// the classes along m, so that a lane holds four consecutive classes of one
// row. Nothing of them leaves the workgroup but
//   forward   per row and tile the maximum, the sum of exponentials around it
//             and the target's logit;
//   backward  G = S * grad * (exp(l - lse) - [v == target]), rounded once to
//             the type of x, and what that rounding took from the target's
//             entry: G's largest entry of a row is usually that one, and its
//             error alone would be the same relative error in all of dx and dw.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../xent.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// exp(a) for a <= 0 or moderate: one multiplication and the hardware's exp2
__device__ __forceinline__ float fast_exp(float a) { return __builtin_amdgcn_exp2f(a * kLog2e); }

// w's and x's rows are whole granules (K-contiguous operands)
template <typename T, typename C>
__global__ __launch_bounds__(C::threads) void xent_loss_kernel(const LossArgs a, int tiles_m, int tiles_n)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    constexpr int KI = 128 / int(sizeof(T));
    int tm, tn;
    strip_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = int64_t(tm) * C::BM, n0 = int64_t(tn) * C::BN;
    floatx4_t acc[C::FM][C::FN];
    NoExtra none;
    tile_product<T, C, false, false>(GemmOperand{a.r.w, a.r.ldw, a.V, a.Dp}, GemmOperand{a.r.x, a.r.ldx, a.N, a.Dp},
                                     m0, n0, 0, int((a.Dp + KI - 1) / KI), smem, acc, none);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % C::WM, wn = wave / C::WM;
    const int mw = wm * (C::BM / C::WM) + (lane >> 4) * 4;      // first class of this lane in the tile
    float2 *red = reinterpret_cast<float2 *>(smem);             // [WM][BN]
    const int left = int(min(int64_t(C::BM), a.V - m0)) - mw;   // classes of this lane that exist
    if (m0 + C::BM > a.V) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (i * 16 + v >= left) acc[i][j][v] = -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int col = wn * (C::BN / C::WN) + 16 * j + (lane & 15);
        const int64_t row = n0 + col;
        const int64_t t = row < a.N ? a.target[row] - m0 - mw : -1;   // among this lane's classes: 16i + v
        if (__ballot(t >= 0 && t < C::FM * 16 && t < left && (t & 15) < 4)) {
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (t == i * 16 + v && i * 16 + v < left) a.loss[row] = acc[i][j][v];
        }
        float m = acc[0][j][0];
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) m = fmaxf(m, acc[i][j][v]);
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float mm = m == -__builtin_inff() ? 0.f : m;      // no class here: exp(-inf) = 0 below
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][v], kLog2e, mm * -kLog2e));
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (lane < 16) red[wm * C::BN + col] = float2{m, s};
    }
    __syncthreads();
    for (int col = threadIdx.x; col < C::BN && n0 + col < a.N; col += C::threads) {
        float m = red[col].x;
#pragma unroll
        for (int w = 1; w < C::WM; ++w) m = fmaxf(m, red[w * C::BN + col].x);
        const float mm = m == -__builtin_inff() ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < C::WM; ++w) s += red[w * C::BN + col].y * fast_exp(red[w * C::BN + col].x - mm);
        a.partial[int64_t(tm) * a.N + n0 + col] = float2{m, s};
    }
}

template <typename T, typename C>
__global__ __launch_bounds__(C::threads) void xent_g_kernel(const GradArgs a, int tiles_m, int tiles_n)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    constexpr int KI = 128 / int(sizeof(T));
    int tm, tn;
    strip_tile(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = int64_t(tm) * C::BM, n0 = int64_t(tn) * C::BN;
    floatx4_t acc[C::FM][C::FN];
    NoExtra none;
    const char *w = static_cast<const char *>(a.r.w) + a.v0 * a.r.ldw;
    tile_product<T, C, false, false>(GemmOperand{w, a.r.ldw, a.P, a.Dp}, GemmOperand{a.r.x, a.r.ldx, a.N, a.Dp}, m0,
                                     n0, 0, int((a.Dp + KI - 1) / KI), smem, acc, none);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % C::WM, wn = wave / C::WM;
    const int mw = wm * (C::BM / C::WM) + (lane >> 4) * 4;
    const int left = int(min(int64_t(C::BM), a.P - m0)) - mw;
    const float S = a.scale ? a.scale[0] : 1.f;
    const int64_t nw = n0 + wn * (C::BN / C::WN);
    if constexpr (sizeof(T) == 2) {
        // which 32 x 32 blocks of G hold a target
        const int64_t cw = a.v0 + m0 + wm * (C::BM / C::WM);
#pragma unroll
        for (int r = 0; r < C::FN / 2; ++r) {
            const int64_t c = a.t32[nw + 32 * r + (lane & 31)] - cw;
#pragma unroll
            for (int b = 0; b < C::FM / 2; ++b) {
                const bool any = __ballot(c >= 32 * b && c < 32 * b + 32) != 0;
                if (lane == 0)
                    a.hits[((m0 + wm * (C::BM / C::WM)) / 32 + b) * a.ldh + nw / 32 + r] = any ? 1 : 0;
            }
        }
    }
    const bool edge = m0 + C::BM > a.P;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int64_t row = nw + 16 * j + (lane & 15);   // below rows_pad
        const int t = a.t32[row];
        const bool ok = t >= 0;
        const float gs = ok ? a.grad[row] * S : 0.f, c = ok ? a.lse[row] * -kLog2e : 0.f;
        T *g = static_cast<T *>(a.g) + row * a.ldg + m0 + mw;
        // exp(l - lse) as one fma and exp2: the rounding of lse * log2(e) is of
        // the size of lse's own
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                acc[i][j][v] = gs * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][v], kLog2e, c));
        if (__ballot(!ok) || edge) {
            // masked rows and classes past the end: selected away, never multiplied
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = ok && i * 16 + v < left ? acc[i][j][v] : 0.f;
        }
        const int64_t tl = ok ? t - a.v0 - m0 - mw : -1;
        if (__ballot(tl >= 0 && tl < C::FM * 16 && (tl & 15) < 4)) {
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (tl == i * 16 + v) {
                        acc[i][j][v] -= gs;
                        if constexpr (sizeof(T) == 2)
                            static_cast<T *>(a.low)[row] =
                                T(acc[i][j][v] - static_cast<float>(T(acc[i][j][v])));
                    }
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const float q[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            store_vec<4>(g + i * 16, q);
        }
    }
}

template <typename C, typename K, typename A>
hipError_t launch_tiles(K kernel, const A &a, int64_t M, int64_t N, hipStream_t s)
{
    const int64_t tm = (M + C::BM - 1) / C::BM, tn = (N + C::BN - 1) / C::BN;
    if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, C::lds_bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(unsigned(tm * tn)), dim3(C::threads), C::lds_bytes, s, a, int(tm), int(tn));
    return hipGetLastError();
}

using C256 = TileCfg<256, 256, 2, 4, 2>;
using C128 = TileCfg<128, 128, 2, 2, 2>;
using C64 = TileCfg<64, 64, 2, 2, 3>;
using CNarrow = TileCfg<128, 16, 4, 1, 4>;

template <typename T>
hipError_t loss_tile(const LossArgs &a, int tile, hipStream_t s)
{
    switch (tile) {
    case kTile256: return launch_tiles<C256>(xent_loss_kernel<T, C256>, a, a.V, a.N, s);
    case kTile128: return launch_tiles<C128>(xent_loss_kernel<T, C128>, a, a.V, a.N, s);
    case kTile64: return launch_tiles<C64>(xent_loss_kernel<T, C64>, a, a.V, a.N, s);
    default: return launch_tiles<CNarrow>(xent_loss_kernel<T, CNarrow>, a, a.V, a.N, s);
    }
}

template <typename T>
hipError_t g_tile(const GradArgs &a, int tile, hipStream_t s)
{
    switch (tile) {
    case kTile256: return launch_tiles<C256>(xent_g_kernel<T, C256>, a, a.P, a.N, s);
    case kTile128: return launch_tiles<C128>(xent_g_kernel<T, C128>, a, a.P, a.N, s);
    default: return launch_tiles<C64>(xent_g_kernel<T, C64>, a, a.P, a.N, s);
    }
}

}  // namespace

hipError_t launch_xent_loss(const LossArgs &a, int dtype, int tile, hipStream_t s)
{
    if (dtype == 0) return loss_tile<float>(a, tile, s);
    if (dtype == 1) return loss_tile<_Float16>(a, tile, s);
    return loss_tile<__bf16>(a, tile, s);
}

hipError_t launch_xent_g(const GradArgs &a, int dtype, int tile, hipStream_t s)
{
    if (dtype == 0) return g_tile<float>(a, tile, s);
    if (dtype == 1) return g_tile<_Float16>(a, tile, s);
    return g_tile<__bf16>(a, tile, s);
}

}  // namespace im2win
