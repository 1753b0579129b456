// Logit tiles of the linear cross entropy: l[n][v] = sum_d w[v][d] x[n][d], with
// the classes along m, so that a lane holds four consecutive classes of one
// row. Nothing of them leaves the workgroup but
//   forward   per row and tile the maximum, the sum of exponentials around it
//             and the target's logit;
//   backward  G = S * grad * (exp(l - lse) - [v == target]), rounded once to
//             the type of x, and in half precision what that rounding took:
//             from the target's entry (G's largest entry of a row is usually
//             that one, and its error alone would be the same relative error
//             in all of dx and dw), and summed over the others of each wave's
//             classes (sum_v G is 0, so that a vector which all class weights
//             share is not in dx; with the roundings it would be, times their
//             sum). That sum is formed only where class weights share
//             something: G of 16384 classes then takes 0.81 ms, else 0.80.
// Bound by the matrix cores (many rows) or by the one read of w (few). 8192 rows,
// 131072 classes, 4096 features, bf16: the losses in 6.2 ms, 1410 TFLOP/s (the
// library's plain product of these operands 1450), G of 16384 classes 0.80 ms,
// 1370; 1 row, 65536 classes, 2048 features 61 us, 4.4 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../xent.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// exp(a) for a <= 0 or moderate: one multiplication and the hardware's exp2
__device__ __forceinline__ float fast_exp(float a) { return __builtin_amdgcn_exp2f(a * kLog2e); }

// exp(l - b) as exp2(fma(l, log2 e, -b log2 e)), one fma per logit: the rounding of
// b log2 e (3e-6 of the result for b = 40) is the same for a row's logits, and this
// factor takes it out again once per row
__device__ __forceinline__ float rounding_of(float b)
{
    return __builtin_amdgcn_exp2f(-__builtin_fmaf(b, kLog2e, b * -kLog2e));
}

// Whether some lane's b is so large that the rounding of b log2 e is no small number
// (its exp2 loses digits from b = 10^7 on and overflows beyond 10^9): then b is
// taken from the logits first, which is exact where it matters (logits within a
// factor of two of b). The comparison is one per row and tile (4097 rows, 50001
// classes, 1032 features, fp16: losses 446 -> 448.6 us).
__device__ __forceinline__ bool large(float b) { return __ballot(fabsf(b) > 1048576.f) != 0; }

// the tile pipelines of the logits: w's and x's rows are whole granules; a
// workgroup takes every gridDim.x-th tile
template <typename T, typename C>
struct LogitTiles {
    TilePipe<T, C, false, false> pipe;
    GemmOperand w, x;
    int tiles_m, tiles_n, stages;
    int64_t m0, n0;          // of the tile that run() is to multiply

    __device__ __forceinline__ LogitTiles(char *smem, const XentRows &r, int64_t v0, int64_t V, int64_t N, int64_t Dp,
                                          int tm, int tn)
        : pipe(smem), w{static_cast<const char *>(r.w) + v0 * r.ldw, r.ldw, V, Dp}, x{r.x, r.ldx, N, Dp}, tiles_m(tm),
          tiles_n(tn), stages(int((Dp + pipe.KI - 1) / pipe.KI))
    {
    }
    __device__ __forceinline__ void start(int t)
    {
        int tm, tn;
        strip_tile(t, tiles_m, tiles_n, tm, tn);
        m0 = int64_t(tm) * C::BM;
        n0 = int64_t(tn) * C::BN;
        if constexpr (kSplitWaves<C>) {
            const int q = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            pipe.start(w, x, m0, n0, stages * q / C::groups, stages * (q + 1) / C::groups);
        } else {
            pipe.start(w, x, m0, n0, 0, stages);
        }
    }
    // the tile's logits as the epilogue's waves hold them; `next` tiles are
    // started meanwhile where the buffers allow it
    template <int SINCE, typename E>
    __device__ __forceinline__ void run(bool since, int next, char *smem, floatx4_t (&out)[E::FM][E::FN])
    {
        NoExtra none;
        if constexpr (kSplitWaves<C>) {
            floatx4_t acc[C::FM][C::FN];
            pipe.template run<0>(false, acc, none);
            join_waves<C>(smem, acc, out);
        } else {
            pipe.template run<SINCE>(since, out, none);
        }
        if (next < tiles_m * tiles_n) start(next);
    }
};

template <typename T, typename C>
__global__ __launch_bounds__(C::threads, C::per_simd) void xent_loss_kernel(const LossArgs a, int tiles_m, int tiles_n)
{
    using E = typename EpiOf<C>::type;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    float2 *red = reinterpret_cast<float2 *>(smem + C::lds_bytes);   // [WM][BN], beside the stage buffers
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % E::WM, wn = wave / E::WM;
    const int mw = wm * (E::BM / E::WM) + (lane >> 4) * 4;      // first class of this lane in the tile
    const int tiles = tiles_m * tiles_n;
    LogitTiles<T, C> lt(smem, a.r, 0, a.V, a.N, a.Dp, tiles_m, tiles_n);
    lt.start(blockIdx.x);
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t m0 = lt.m0, n0 = lt.n0;
        const int left = int(min(int64_t(E::BM), a.V - m0)) - mw;   // classes of this lane that exist
        // the rows' targets among this lane's classes 16i + v, loaded ahead
        int64_t target[E::FN];
#pragma unroll
        for (int j = 0; j < E::FN; ++j)
            target[j] = a.target[min(n0 + wn * (E::BN / E::WN) + 16 * j + (lane & 15), a.N - 1)];
        floatx4_t acc[E::FM][E::FN];
        lt.template run<0, E>(false, tile + int(gridDim.x), smem, acc);

        if (m0 + E::BM > a.V) {
#pragma unroll
            for (int i = 0; i < E::FM; ++i)
#pragma unroll
                for (int j = 0; j < E::FN; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (i * 16 + v >= left) acc[i][j][v] = -__builtin_inff();
        }
#pragma unroll
        for (int j = 0; j < E::FN; ++j) {
            const int col = wn * (E::BN / E::WN) + 16 * j + (lane & 15);
            const int64_t row = n0 + col, t = row < a.N ? target[j] - m0 - mw : -1;
            if (__ballot(t >= 0 && t < E::FM * 16 && t < left && (t & 15) < 4)) {
#pragma unroll
                for (int i = 0; i < E::FM; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (t == i * 16 + v && i * 16 + v < left) a.loss[row] = acc[i][j][v];
            }
            float m = acc[0][j][0];
#pragma unroll
            for (int i = 0; i < E::FM; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) m = fmaxf(m, acc[i][j][v]);
            m = fmaxf(m, __shfl_xor(m, 16, 64));
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            float mm = m == -__builtin_inff() ? 0.f : m;            // no class here: exp(-inf) = 0 below
            if (large(mm)) {
#pragma unroll
                for (int i = 0; i < E::FM; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] -= mm;
                mm = 0.f;
            }
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < E::FM; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][v], kLog2e, mm * -kLog2e));
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            s *= rounding_of(mm);
            if (lane < 16) red[wm * E::BN + col] = float2{m, s};
        }
        // LDS accesses alone are waited for: the next tile's copies stay in flight.
        // The next writes to red come after the barriers of the next run().
        stage_barrier();
        for (int col = threadIdx.x; col < E::BN && n0 + col < a.N; col += C::threads) {
            float m = red[col].x;
#pragma unroll
            for (int w = 1; w < E::WM; ++w) m = fmaxf(m, red[w * E::BN + col].x);
            const float mm = m == -__builtin_inff() ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < E::WM; ++w) s += red[w * E::BN + col].y * fast_exp(red[w * E::BN + col].x - mm);
            a.partial[m0 / E::BM * a.N + n0 + col] = float2{m, s};
        }
    }
}

template <typename T, typename C>
__global__ __launch_bounds__(C::threads, C::per_simd) void xent_g_kernel(const GradArgs a, int tiles_m, int tiles_n)
{
    using E = typename EpiOf<C>::type;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    constexpr bool PAIRS = sizeof(T) == 2 && E::FM % 2 == 0;
    constexpr int STORES = PAIRS ? E::FM * E::FN / 2 : E::FM * E::FN;   // of a wave and tile
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % E::WM, wn = wave / E::WM;
    const int mw = wm * (E::BM / E::WM) + (lane >> 4) * 4;
    const int tiles = tiles_m * tiles_n;
    const float S = a.scale ? a.scale[0] : 1.f;
    constexpr bool HALF = sizeof(T) == 2;
    LogitTiles<T, C> lt(smem, a.r, a.v0, a.P, a.N, a.Dp, tiles_m, tiles_n);
    lt.start(blockIdx.x);
    bool some = false;                         // weights of either sign, the usual case, need no rest
    if constexpr (HALF) {
        for (int f = lane; f < a.somes; f += 64) some |= a.some[f] != 0;
        some = __ballot(some) != 0;
    }
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t m0 = lt.m0, n0 = lt.n0, nw = n0 + wn * (E::BN / E::WN);
        const int left = int(min(int64_t(E::BM), a.P - m0)) - mw;
        // of the rows of this lane's columns (below rows_pad), loaded ahead
        int target[E::FN];
        float grad[E::FN], lse[E::FN];
#pragma unroll
        for (int j = 0; j < E::FN; ++j) {
            const int64_t row = nw + 16 * j + (lane & 15), in = min(row, a.N - 1);
            target[j] = a.t32[row];
            grad[j] = a.grad[in];
            lse[j] = a.lse[in];
        }
        floatx4_t acc[E::FM][E::FN];
        lt.template run<STORES, E>(tile != int(blockIdx.x), tile + int(gridDim.x), smem, acc);

        if constexpr (sizeof(T) == 2) {
            // which 32 x 32 blocks of G hold a target
            const int64_t cw = a.v0 + m0 + wm * (E::BM / E::WM);
            if constexpr (E::FN == 1) {
                // a block's rows are shared by waves: each sees all 32 of them, the
                // first wave of each block of classes writes
                static_assert(E::BN == 32 && (E::FM == 1 || E::FM == 2), "one block of rows");
                const int64_t b32 = m0 + wm * (E::BM / E::WM) / 32 * 32, c = a.t32[n0 + (lane & 31)] - a.v0 - b32;
                const bool any = __ballot(c >= 0 && c < 32) != 0;
                if (lane == 0 && wn == 0) a.hits[b32 / 32 * a.ldh + n0 / 32] = any ? 1 : 0;
            }
#pragma unroll
            for (int r = 0; r < E::FN / 2; ++r) {
                const int64_t c0 = target[2 * r] - cw, c1 = target[2 * r + 1] - cw;
#pragma unroll
                for (int b = 0; b < E::FM / 2; ++b) {
                    const bool any = __ballot((c0 >= 32 * b && c0 < 32 * b + 32) ||
                                              (c1 >= 32 * b && c1 < 32 * b + 32)) != 0;
                    if (lane == 0)
                        a.hits[((m0 + wm * (E::BM / E::WM)) / 32 + b) * a.ldh + nw / 32 + r] = any ? 1 : 0;
                }
            }
        }
        const bool edge = m0 + E::BM > a.P;
#pragma unroll
        for (int j = 0; j < E::FN; ++j) {
            const int64_t row = nw + 16 * j + (lane & 15);
            const int t = target[j];
            const bool ok = t >= 0;
            float b = ok ? lse[j] : 0.f;
            if (large(b)) {
#pragma unroll
                for (int i = 0; i < E::FM; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] -= b;
                b = 0.f;
            }
            const float gs = ok ? grad[j] * S : 0.f, c = b * -kLog2e;
            const float ps = ok ? gs * rounding_of(b) : 0.f;
#pragma unroll
            for (int i = 0; i < E::FM; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[i][j][v] = ps * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][v], kLog2e, c));
            if (__ballot(!ok) || edge) {
                // masked rows and classes past the end: selected away, never multiplied
#pragma unroll
                for (int i = 0; i < E::FM; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = ok && i * 16 + v < left ? acc[i][j][v] : 0.f;
            }
            float rest = 0.f;
            const int64_t tl = ok ? t - a.v0 - m0 - mw : -1;
            if (__ballot(tl >= 0 && tl < E::FM * 16 && (tl & 15) < 4)) {
#pragma unroll
                for (int i = 0; i < E::FM; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (tl == i * 16 + v) {
                            acc[i][j][v] -= gs;
                            if constexpr (HALF) {
                                const T low = T(acc[i][j][v] - static_cast<float>(T(acc[i][j][v])));
                                static_cast<T *>(a.low)[row] = low;
                                rest = -static_cast<float>(low);
                            }
                        }
            }
            if (HALF && some) {
#pragma unroll
                for (int i = 0; i < E::FM; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) rest += acc[i][j][v] - static_cast<float>(T(acc[i][j][v]));
                rest += __shfl_xor(rest, 16, 64);
                rest += __shfl_xor(rest, 32, 64);
                if (lane < 16) a.rest[(m0 / E::BM * E::WM + wm) * a.ldr + row] = rest;
            }
            T *g = static_cast<T *>(a.g) + row * a.ldg + m0;
            if constexpr (PAIRS) {
                const int m8 = wm * (E::BM / E::WM) + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
#pragma unroll
                for (int i = 0; i < E::FM; i += 2) *reinterpret_cast<uint4 *>(g + m8 + i * 16) =
                    pair_blocks<T>(acc[i][j], acc[i + 1][j]);
            } else {
#pragma unroll
                for (int i = 0; i < E::FM; ++i) {
                    const float q[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    store_vec<4>(g + mw + i * 16, q);
                }
            }
        }
    }
}

template <typename C, typename K, typename A>
hipError_t launch_tiles(K kernel, int lds, std::atomic<uint64_t> &allowed, const A &a, int64_t stages,
                        int64_t M, int64_t N, hipStream_t s)
{
    const int64_t tm = (M + C::BM - 1) / C::BM, tn = (N + C::BN - 1) / C::BN;
    if (tm * tn > kMaxTiles) return hipErrorInvalidValue;
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), lds, allowed);
    if (e != hipSuccess) return e;
    // C32K joins its waves in the stage buffers: a workgroup per tile
    const int64_t grid = kSplitWaves<C> ? std::min(tm * tn, max_groups(C::threads)) : grid_of<C>(tm * tn, stages);
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(C::threads), lds, s, a, int(tm), int(tn));
    return hipGetLastError();
}

template <typename T>
hipError_t loss_tile(const LossArgs &a, int tile, hipStream_t s)
{
    static std::atomic<uint64_t> allowed[kTiles];
    const int64_t stages = (a.Dp * int64_t(sizeof(T)) + 127) / 128;
    switch (tile) {
    case kTile256: return launch_tiles<C256>(xent_loss_kernel<T, C256>, C256::lds_bytes + C256::WM * C256::BN * 8, allowed[kTile256], a, stages, a.V, a.N, s);
    case kTile128: return launch_tiles<C128>(xent_loss_kernel<T, C128>, C128::lds_bytes + C128::WM * C128::BN * 8, allowed[kTile128], a, stages, a.V, a.N, s);
    case kTile64x32:
        return launch_tiles<C64x32>(xent_loss_kernel<T, C64x32>, C64x32::lds_bytes + 2 * 32 * 8, allowed[kTile64x32], a, stages, a.V,
                                    a.N, s);
    case kTile32K:
        return launch_tiles<C32K>(xent_loss_kernel<T, C32K>, C32K::lds_bytes + 2 * 32 * 8, allowed[kTile32K], a, stages, a.V, a.N, s);
    case kTile64: return launch_tiles<C64>(xent_loss_kernel<T, C64>, C64::lds_bytes + C64::WM * C64::BN * 8, allowed[kTile64], a, stages, a.V, a.N, s);
    default: return launch_tiles<CNarrow>(xent_loss_kernel<T, CNarrow>, CNarrow::lds_bytes + CNarrow::WM * CNarrow::BN * 8, allowed[kTileNarrow], a, stages, a.V, a.N, s);
    }
}

template <typename T>
hipError_t g_tile(const GradArgs &a, int tile, hipStream_t s)
{
    static std::atomic<uint64_t> allowed[kTiles];
    const int64_t stages = (a.Dp * int64_t(sizeof(T)) + 127) / 128;
    switch (tile) {
    case kTile256: return launch_tiles<C256>(xent_g_kernel<T, C256>, C256::lds_bytes, allowed[kTile256], a, stages, a.P, a.N, s);
    case kTile128: return launch_tiles<C128>(xent_g_kernel<T, C128>, C128::lds_bytes, allowed[kTile128], a, stages, a.P, a.N, s);
    case kTile32K:
        // the products read G in whole stages of 64: the padding is written too
        return launch_tiles<C32K>(xent_g_kernel<T, C32K>, C32K::lds_bytes, allowed[kTile32K], a, stages, (a.P + 63) / 64 * 64,
                                  (a.N + 63) / 64 * 64, s);
    case kTile64x32:
        return launch_tiles<C64x32>(xent_g_kernel<T, C64x32>, C64x32::lds_bytes, allowed[kTile64x32], a, stages, a.P,
                                    (a.N + 63) / 64 * 64, s);
    default: return launch_tiles<C64>(xent_g_kernel<T, C64>, C64::lds_bytes, allowed[kTile64], a, stages, a.P, a.N, s);
    }
}

}  // namespace

int64_t rest_blocks(int tile, int64_t P)
{
    const auto blocks = [](int64_t m, int64_t BM, int64_t WM) { return (m + BM - 1) / BM * WM; };
    switch (tile) {
    case kTile256: return blocks(P, C256::BM, C256::WM);
    case kTile128: return blocks(P, C128::BM, C128::WM);
    case kTile32K: return blocks((P + 63) / 64 * 64, C32K::BM, C32K::Epi::WM);
    case kTile64x32: return blocks(P, C64x32::BM, C64x32::WM);
    default: return blocks(P, C64::BM, C64::WM);
    }
}

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
