// The feed-forward block's plain products, each output's contiguous index along m:
//   y[n][o]  = sum_f Wd[o][f] h[n][f]                        both in rows
//   dx[n][d] = sum_f Wg[f][d] da[n][f] + Wu[f][d] du[n][f]   weights in columns, G in
//              rows, one accumulation over the two segments of K
//   dWd[o][f] = sum_n h[n][f] dy[n][o]                       both in columns
//   dWg[f][d], dWu[f][d] = sum_n x[n][d] da[n][f], .. du     both in columns, the two
//              outputs as one launch's tiles
// K may be split over workgroups into fp32 slabs that another kernel adds in order.
// Bound by the matrix cores: 8192 rows, 4096 inputs and outputs, 16384 hidden features,
// bf16: y 903 us (1217 TFLOP/s), dx 1562 (1408), dWd 835 (1317), dWg and dWu 1730 (1271).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ff_common.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

// tiles begin, begin + step, .. of one product
template <typename T, typename C, bool ACOLS, bool BCOLS>
__device__ __forceinline__ void product_tiles(const FfProduct &a, int tiles_m, int tiles_n, int begin, int step,
                                              char *smem)
{
    constexpr int KI = 128 / int(sizeof(T));
    constexpr bool HALF = sizeof(T) == 2, SCALED = std::is_same<T, _Float16>::value;
    constexpr int STORES = HALF ? C::FM * C::FN / 2 : C::FM * C::FN;    // of a wave and whole tile, at least
    // tiles_n: of all outputs
    const int tiles = tiles_m * tiles_n, all = tiles * a.split, per_out = tiles_n / a.outs;
    const int nk = int((a.K + KI - 1) / KI);               // stages of a segment
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % C::WM, wn = wave / C::WM;
    const int mw = wm * (C::BM / C::WM), nw = wn * (C::BN / C::WN);
    const float inv = a.amax ? 1.f / (dy_scale(a.amax) * x_scale(a.amax)) : 1.f;
    TilePipe<T, C, ACOLS, BCOLS> pipe(smem);
    int part = 0, o = 0;
    int64_t m0 = 0, n0 = 0;
    // stages of segment g in this part of K
    auto first_of = [&](int g) { return max(0, int(int64_t(nk) * a.segs * part / a.split) - g * nk); };
    auto end_of = [&](int g) { return min(nk, int(int64_t(nk) * a.segs * (part + 1) / a.split) - g * nk); };
    auto start_seg = [&](int g) {
        const GemmOperand A{g ? a.a[1] : a.a[0], g ? a.lda[1] : a.lda[0], a.a_count, a.k_a};
        const GemmOperand B{static_cast<const char *>(a.b) + (g + o) * a.b_step, a.ldb, a.b_count, a.k_b};
        pipe.start(A, B, m0, n0, first_of(g), end_of(g));
    };
    int seg = 0;                               // that the pipe has started
    auto start = [&](int t) {
        int tm, tn;
        part = t / tiles;
        strip_tile(t - part * tiles, tiles_m, tiles_n, tm, tn);
        o = tn / per_out;
        m0 = int64_t(tm) * C::BM;
        n0 = int64_t(tn - o * per_out) * C::BN;
        seg = a.segs > 1 && first_of(0) >= end_of(0) ? 1 : 0;
        start_seg(seg);
    };
    // products of two operands in columns with the largest tile have no registers
    // left for the next tile's addresses: their launch has a workgroup for every tile
    constexpr bool ONE = ACOLS && BCOLS && HALF && C::FM == 8;
    start(begin);
    bool stored = false;                       // the last epilogue stored a whole tile
    for (int t = begin; t < all; t += ONE ? all : step) {
        floatx4_t acc[C::FM][C::FN];
        bool clear = true;
        for (;;) {
            NoExtra none;
            pipe.template run<STORES>(stored, acc, none, clear);
            if (seg + 1 >= a.segs || first_of(seg + 1) >= end_of(seg + 1)) break;
            start_seg(++seg);
            clear = stored = false;
        }
        const int cur = part, co = o;
        const int64_t mt = m0 + mw, nt = n0 + nw;
        if constexpr (!ONE) {
            stored = m0 + C::BM <= a.M && n0 + C::BN <= a.n;
            if (t + step < all) start(t + step);
        }
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int64_t row = nt + 16 * j + (lane & 15);
            if (row >= a.n) continue;
            if (a.slab) {
                float *p = a.slab + ((int64_t(cur) * a.outs + co) * a.n + row) * a.M;
#pragma unroll
                for (int i = 0; i < C::FM; ++i) {
                    const int64_t m = mt + i * 16 + (lane >> 4) * 4;
                    const float q[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    store_some<4>(p + m, a.M - m, q);
                }
                continue;
            }
            T *p = static_cast<T *>(co ? a.out[1] : a.out[0]) + row * a.ldo;
            float by = inv;
            if constexpr (SCALED)
                if (a.scale) by = 1.f / a.scale[row];
#pragma unroll
            for (int i = 0; i < C::FM; ++i) acc[i][j] *= by;
            if constexpr (HALF) {
                const int64_t m8 = mt + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
#pragma unroll
                for (int i = 0; i < C::FM; i += 2) {
                    const uint4 q = pair_blocks<T>(acc[i][j], acc[i + 1][j]);
                    store_some_raw(p + m8 + i * 16, a.M - m8 - i * 16, __builtin_bit_cast(Raw<T, 8>, q));
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::FM; ++i) {
                    const int64_t m = mt + i * 16 + (lane >> 4) * 4;
                    const float q[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    store_some<4>(p + m, a.M - m, q);
                }
            }
        }
    }
}

template <typename T, typename C, bool ACOLS, bool BCOLS>
__global__ __launch_bounds__(C::threads, C::per_simd) void ff_product_kernel(const FfProduct a, int tiles_m, int tiles_n)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    product_tiles<T, C, ACOLS, BCOLS>(a, tiles_m, tiles_n, blockIdx.x, gridDim.x, smem);
}

struct FfTiles {
    int m, n, all;           // tiles along m and n (of all outputs), workgroups
};

// The products of a backward pass in one launch, a workgroup per tile, the longest first:
// none fills the chip by itself (or its last round does not), and all need only da, du
// and h. 4097 x 1032 x 3001, fp16: 173 us, 242 one after the other.
template <typename T, typename C>
__global__ __launch_bounds__(C::threads, C::per_simd) void ff_all_kernel(const FfProduct dx, const FfProduct dwd,
                                                                         const FfProduct dwgu, FfTiles tx, FfTiles td,
                                                                         FfTiles tg)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int b = blockIdx.x;
    if (b < tx.all)
        product_tiles<T, C, true, false>(dx, tx.m, tx.n, b, tx.all, smem);
    else if (b < tx.all + tg.all)
        product_tiles<T, C, true, true>(dwgu, tg.m, tg.n, b - tx.all, tg.all, smem);
    else
        product_tiles<T, C, true, true>(dwd, td.m, td.n, b - tx.all - tg.all, td.all, smem);
}

template <typename C>
FfTiles tiles_of(const FfProduct &a)
{
    const int64_t m = ceil_div(a.M, C::BM), n = ceil_div(a.n, C::BN) * a.outs;
    return {int(m), int(n), m * n * a.split > kMaxTiles ? -1 : int(m * n * a.split)};
}

template <typename T, typename C, bool ACOLS, bool BCOLS>
hipError_t launch_tiles(const FfProduct &a, hipStream_t s)
{
    constexpr bool ONE = ACOLS && BCOLS && sizeof(T) == 2 && C::FM == 8;    // a workgroup for every tile
    const auto kernel = ff_product_kernel<T, C, ACOLS, BCOLS>;
    const FfTiles t = tiles_of<C>(a);
    if (t.all < 0 || (ONE && t.all > max_groups(C::threads))) return hipErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), C::lds_bytes, allowed);
    if (e != hipSuccess) return e;
    const int64_t stages = ceil_div(a.K * int64_t(sizeof(T)), 128) * a.segs / a.split;
    const int64_t grid = ONE ? t.all : grid_of<C>(t.all, stages);
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(C::threads), C::lds_bytes, s, a, t.m, t.n);
    return hipGetLastError();
}

template <bool ACOLS, bool BCOLS>
hipError_t launch_product(const FfProduct &p, int dtype, int tile, hipStream_t s)
{
    return with_ff_type(dtype, [&](auto t) {
        using T = decltype(t);
        switch (tile) {
        case kTile256: return launch_tiles<T, C256, ACOLS, BCOLS>(p, s);
        case kTile128: return launch_tiles<T, C128, ACOLS, BCOLS>(p, s);
        default: return launch_tiles<T, C64, ACOLS, BCOLS>(p, s);
        }
    });
}

// The slabs added in a fixed order: a workgroup takes 256 / Q chunks of 4 outputs, Q threads
// a chunk, thread q slabs q, q + Q, .. (few outputs and many slabs would leave most of the
// chip idle: 64 x 512 outputs in 16 slabs, fp32, 6.9 us with one thread a chunk)
struct FfJoin {
    FfProduct p[3];
    int64_t end[3];          // chunks up to and with a product's
    int count;
    const float *amax;       // of those products that are scaled
};
template <typename T, int Q>
__global__ __launch_bounds__(256) void ff_join_kernel(const FfJoin j)
{
    __shared__ float4 sum[Q > 1 ? 256 : 1];
    constexpr int CH = 256 / Q;
    const int64_t step = int64_t(gridDim.x) * CH, total = j.end[j.count - 1];
    const float inv = j.amax ? 1.f / (dy_scale(j.amax) * x_scale(j.amax)) : 1.f;
    const int t = threadIdx.x % CH, q = threadIdx.x / CH;
    for (int64_t i0 = int64_t(blockIdx.x) * CH; i0 < total; i0 += step) {
        const int64_t i = min(i0 + t, total - 1);
        int k = 0;
        while (k + 1 < j.count && i >= j.end[k]) ++k;
        const FfProduct &a = j.p[k];
        const int64_t chunks = (a.M + 3) / 4, c = i - (k ? j.end[k - 1] : 0);
        const int64_t r = c / chunks, m = (c - r * chunks) * 4, left = a.M - m;
        const int64_t part = a.outs * a.n * a.M;
        const float *src = a.slab + r * a.M + m;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (left >= 4) {
#pragma unroll 4
            for (int p = q; p < a.split; p += Q) {
                float g[4];
                load_vec<4>(src + p * part, g);
#pragma unroll
                for (int v = 0; v < 4; ++v) f[v] += g[v];
            }
        } else {
            for (int p = q; p < a.split; p += Q)
                for (int v = 0; v < left; ++v) f[v] += src[p * part + v];
        }
        if constexpr (Q > 1) {
            __syncthreads();
            sum[threadIdx.x] = float4{f[0], f[1], f[2], f[3]};
            __syncthreads();
            if (q > 0) continue;
#pragma unroll
            for (int p = 1; p < Q; ++p) {
                const float4 g = sum[p * CH + t];
                f[0] += g.x;
                f[1] += g.y;
                f[2] += g.z;
                f[3] += g.w;
            }
        }
        if (i0 + t >= total) continue;
        if (a.amax || a.scale) {
            const float by = a.scale ? 1.f / a.scale[r] : inv;
#pragma unroll
            for (int v = 0; v < 4; ++v) f[v] *= by;
        }
        const int o = int(r / a.n);
        store_some<4>(static_cast<T *>(o ? a.out[1] : a.out[0]) + (r - o * a.n) * a.ldo + m, left, f);
    }
}

}  // namespace

hipError_t launch_ff_y(const FfProduct &p, int dtype, int tile, hipStream_t s)
{
    return launch_product<false, false>(p, dtype, tile, s);
}

hipError_t launch_ff_dx(const FfProduct &p, int dtype, int tile, hipStream_t s)
{
    return launch_product<true, false>(p, dtype, tile, s);
}

hipError_t launch_ff_dw(const FfProduct &p, int dtype, int tile, hipStream_t s)
{
    return launch_product<true, true>(p, dtype, tile, s);
}

hipError_t launch_ff_all(const FfProduct &dx, const FfProduct &dwd, const FfProduct &dwgu, int dtype, int tile,
                         hipStream_t s)
{
    return with_ff_type(dtype, [&](auto t) {
        const auto launch = [&](auto cfg) {
            using C = decltype(cfg);
            const auto kernel = ff_all_kernel<decltype(t), C>;
            const FfTiles x = tiles_of<C>(dx), d = tiles_of<C>(dwd), g = tiles_of<C>(dwgu);
            const int64_t grid = int64_t(x.all) + d.all + g.all;
            if (x.all < 0 || d.all < 0 || g.all < 0 || grid > max_groups(C::threads)) return hipErrorInvalidValue;
            static std::atomic<uint64_t> allowed{0};
            const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), C::lds_bytes, allowed);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(C::threads), C::lds_bytes, s, dx, dwd, dwgu, x, d, g);
            return hipGetLastError();
        };
        return tile == kTile128 ? launch(C128{}) : launch(C64{});
    });
}

hipError_t launch_ff_join(const FfProduct *p, int count, int dtype, hipStream_t s)
{
    FfJoin j{};
    j.count = count;
    int64_t n = 0;
    for (int k = 0; k < count; ++k) {
        j.p[k] = p[k];
        if (p[k].amax) j.amax = p[k].amax;
        n += p[k].outs * p[k].n * ceil_div(p[k].M, 4);
        j.end[k] = n;
    }
    bool many = n < 65536;                     // slabs of few chunks: 8 threads a chunk
    for (int k = 0; k < count; ++k) many = many && p[k].split >= 8;
    const int64_t grid = std::min<int64_t>(ceil_div(n, many ? 32 : 256), 8192);
    return with_ff_type(dtype, [&](auto t) {
        if (many)
            hipLaunchKernelGGL((ff_join_kernel<decltype(t), 8>), dim3(unsigned(grid)), dim3(256), 0, s, j);
        else
            hipLaunchKernelGGL((ff_join_kernel<decltype(t), 1>), dim3(unsigned(grid)), dim3(256), 0, s, j);
        return hipGetLastError();
    });
}

}  // namespace im2win
