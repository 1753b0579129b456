// The gradient products of the linear cross entropy, with the features along m
// (the contiguous index of dx and dw):
//   dx[n][d] = sum_v w[v][d] G[n][v]     G in rows, w in columns
//   dw[v][d] = sum_n x[n][d] G[n][v]     both in columns
// K may be split over workgroups into fp32 slabs that another kernel adds in
// order. In half precision what rounding took from G at each row's target goes
// back in: dx in the epilogue (+ low[n] w[target[n]]), dw as further products
// of the stages in which a row's target is one of the wave's classes (at most
// one more per block of 16 classes, and a block is skipped unless a
// target falls into it). What it took from a row's other entries, summed, goes into dx
// times what the class weights share, c: the roundings then multiply w - c, and an
// offset of all classes cancels as it should, for sum_v G is 0 (30 classes that share
// 64 times their spread, bf16: dx was off by 0.4 of its size). Bound by the matrix
// cores: with 8192 rows, a piece of 16384 classes and 4096 features, bf16, dx takes 0.82
// ms (1340 TFLOP/s) and dw 0.94 ms (1170; 0.90 without hits: both operands come through
// transposed reads, two for each one of rows, and with a workgroup per tile nothing
// covers a tile's first copies and epilogue).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../xent.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

// dw: the products that add low[n] x[n] to the target's class of each row n. With
// many classes few stages have any; with few, every stage has, and what they cost
// is the wait for the rows' targets (1634 rows, 208 classes, 376 features, bf16:
// step 59 us with the targets and lows loaded one after the other when needed, 50
// with both at once and a stage ahead, 34 with K split by the time so measured).
template <typename T, typename C>
struct LowExtra {
    static constexpr int KI = 128 / int(sizeof(T)), KH = KI / 2;
    const ProductArgs &a;
    int64_t c0;              // first class of this wave, relative to the piece
    int s0, nk, lane;
    uint32_t hit = 0;        // bit s & 31: a target of stage s's rows is one of this wave's classes
    // the rows of the stage after a hit are asked for a stage ahead, with small tiles
    // only: their stages are too short to hide the wait (the larger ones lose 8 %,
    // 8192 rows, 1000 classes, 1024 features 137 -> 150 us)
    static constexpr bool AHEAD = C::FM <= 2;
    int next_s = -1;
    uint32_t next = 0;

    // hits of 32 stages at a time: lane l < 32 takes stage l for the first 32
    // classes, the others for the second 32 of a wave of 64 classes
    __device__ __forceinline__ void load_hits(int s)
    {
        uint64_t all = 0;
#pragma unroll
        for (int q = 0; q < (C::FN + 3) / 4; ++q) {
            const int64_t st = (s & ~31) + (lane & 31);
            const bool in = (lane >> 5) * 2 + q * 4 < C::FN && st < nk;
            uint32_t v = 0;
            if (in) {
                const uint8_t *p = a.hits + (c0 / 32 + q * 2 + (lane >> 5)) * a.ldh + st * 2;
                v = p[0] | p[1];
            }
            all |= __ballot(v != 0);
        }
        hit = uint32_t(all) | uint32_t(all >> 32);
    }
    // row s KI + lane: its target among this wave's classes (0xffff: none of them)
    // above the bits of its low
    __device__ __forceinline__ uint32_t row_of(int s) const
    {
        const int64_t r = int64_t(s) * KI + lane;
        const uint32_t t = uint32_t(a.t32[r] - int(a.v0 + c0));
        const uint32_t bits = static_cast<const uint16_t *>(a.low)[r];
        return (t < C::FN * 16 ? t : 0xffffu) << 16 | bits;
    }
    template <typename R>
    __device__ __forceinline__ void run(int s, R read, floatx4_t (&acc)[C::FM][C::FN])
    {
        if ((s & 31) == 0 || s == s0) load_hits(s);
        if (__builtin_expect(!((hit >> (s & 31)) & 1), 1)) return;
        const uint32_t row = s == next_s ? next : row_of(s);
        const int t = int(row >> 16);
        if constexpr (AHEAD) {
            next_s = s + 1;
            next = row_of(min(next_s, nk - 1));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!__ballot((lane / KH) == h && t < C::FN * 16)) continue;
            uint32_t e8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) e8[e] = __shfl(row, h * KH + (lane >> 4) * 8 + e, 64);
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                if (!__ballot((lane / KH) == h && (t >> 4) == j)) continue;
                const uint32_t c = j * 16 + (lane & 15);
                uint32_t f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[e] = (e8[2 * e] >> 16 == c ? e8[2 * e] & 0xffffu : 0u) |
                           (e8[2 * e + 1] >> 16 == c ? e8[2 * e + 1] << 16 : 0u);
                const uint4 b{f[0], f[1], f[2], f[3]};
#pragma unroll
                for (int i = 0; i < C::FM; ++i) acc[i][j] = mfma_half<T>(read(i, h), b, acc[i][j]);
            }
        }
    }
};

// dx: acc += rest * c for this part's share of the blocks of classes, with c what the
// class weights share but no more than the weight of the row's own target (between 0
// and that): then |rest c| is within a rounding of the target's own |G w|, whatever the
// other classes' weights, and no element's error bound grows. (Without it the mean of
// the classes, or the least of those looked at, exceeds an element's bound where the few
// classes that count in its row lie apart from the others.) A lane's column is row n of
// dx; the four lanes of a column take every fourth block.
template <typename T, typename C>
__device__ __forceinline__ void add_rest(const ProductArgs &a, int part, int64_t m0, int64_t n0, int lane,
                                         floatx4_t (&acc)[C::FM][C::FN])
{
    constexpr int E = 16 / int(sizeof(T));
    const int64_t m = m0 + (lane >> 4) * 4;
    // nothing shared (weights of either sign, the usual case): nothing to add
    bool any = false;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        float c[4];
        load_vec<4>(a.shared + m + i * 16, c);
        any |= c[0] != 0.f || c[1] != 0.f || c[2] != 0.f || c[3] != 0.f;
    }
    if (!__ballot(any)) return;
    const int begin = int(int64_t(a.blocks) * part / a.split), end = int(int64_t(a.blocks) * (part + 1) / a.split);
    const int64_t row = n0 + (lane & 15);                // and 16 j on: below ldr, a multiple of 256
    float rest[C::FN];
    int tgt[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        tgt[j] = max(a.t32[row + 16 * j], 0);            // a masked row's rest is 0
        rest[j] = 0.f;
    }
#pragma unroll 2
    for (int b = begin + (lane >> 4); b < end; b += 4)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) rest[j] += a.rest[b * a.ldr + row + 16 * j];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        rest[j] += __shfl_xor(rest[j], 16, 64);
        rest[j] += __shfl_xor(rest[j], 32, 64);
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        float c[4];
        load_vec<4>(a.shared + m + i * 16, c);
        const int64_t at = min(m + i * 16, (a.M + E - 1) / E * E - 4);   // w's rows are whole granules
        Raw<T, 4> w[C::FN];
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            w[j] = load_raw<T, 4>(reinterpret_cast<const T *>(static_cast<const char *>(a.w) + tgt[j] * a.ldw) + at);
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] += rest[j] * __builtin_amdgcn_fmed3f(element(w[j], v), 0.f, c[v]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// tiles begin, begin + step, .. of one product
template <typename T, typename C, bool DW>
__device__ __forceinline__ void product_tiles(const ProductArgs &a, int tiles_m, int tiles_n, int begin, int step,
                                              char *smem)
{
    constexpr int KI = 128 / int(sizeof(T)), E = 16 / int(sizeof(T));   // w's and x's rows are whole granules
    constexpr bool HALF = sizeof(T) == 2;
    constexpr int STORES = HALF ? C::FM * C::FN / 2 : C::FM * C::FN;    // of a wave and whole tile, at least
    const int tiles = tiles_m * tiles_n, all = tiles * a.split;
    const int nk = int((a.K + KI - 1) / KI);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave % C::WM, wn = wave / C::WM;
    const int mw = wm * (C::BM / C::WM), nw = wn * (C::BN / C::WN);
    const float inv = a.scale ? a.scale[1] : 1.f;
    const GemmOperand A{a.a, a.lda, (a.M + E - 1) / E * E, a.k_a};
    const GemmOperand B{a.b, a.ldb, DW ? a.ldb / int64_t(sizeof(T)) : a.n, a.k_b};
    TilePipe<T, C, true, DW> pipe(smem);
    int part = 0;
    int64_t m0 = 0, n0 = 0;
    auto start = [&](int t) {
        int tm, tn;
        part = t / tiles;
        strip_tile(t - part * tiles, tiles_m, tiles_n, tm, tn);
        m0 = int64_t(tm) * C::BM;
        n0 = int64_t(tn) * C::BN;
        pipe.start(A, B, m0, n0, int(int64_t(nk) * part / a.split), int(int64_t(nk) * (part + 1) / a.split));
    };
    // dw in half precision with the largest tile has no registers left for the next
    // tile's addresses: its launch has a workgroup for every tile
    constexpr bool ONE = DW && HALF && C::FM == 8;
    start(begin);
    bool stored = false;                       // the last epilogue stored a whole tile
    for (int t = begin; t < all; t += ONE ? all : step) {
        const int cur = part;
        const int64_t mt = m0 + mw, nt = n0 + nw;
        floatx4_t acc[C::FM][C::FN];
        if constexpr (DW && HALF) {
            LowExtra<T, C> low{a, nt, pipe.s0, nk, lane};
            pipe.template run<STORES>(stored, acc, low);
        } else {
            NoExtra none;
            pipe.template run<STORES>(stored, acc, none);
        }
        if constexpr (HALF && !DW) add_rest<T, C>(a, part, mt, nt, lane, acc);
        if constexpr (!ONE) {
            stored = m0 + C::BM <= a.M && n0 + C::BN <= a.n;
            if (t + step < all) start(t + step);
        }

#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const int64_t row = nt + 16 * j + (lane & 15);
            if (row >= a.n) continue;
            if (a.slab) {
                float *o = a.slab + (int64_t(cur) * a.n + row) * a.M;
#pragma unroll
                for (int i = 0; i < C::FM; ++i) {
                    const int64_t m = mt + i * 16 + (lane >> 4) * 4, left = a.M - m;
                    if (left <= 0) continue;
                    float q[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    if (a.add) {
                        float p[4];
                        load_some<4>(o + m, left, p);
#pragma unroll
                        for (int v = 0; v < 4; ++v) q[v] += p[v];
                    }
                    store_some<4>(o + m, left, q);
                }
                continue;
            }
            int tgt = 0;
            float lv = 0.f;
            if constexpr (!DW) {
                tgt = a.t32[row];
                if (HALF && tgt >= 0) lv = static_cast<float>(static_cast<const T *>(a.low)[row]);
            }
            const T *wt = reinterpret_cast<const T *>(static_cast<const char *>(a.w) + tgt * a.ldw);
            T *o = static_cast<T *>(a.out) + row * a.M;
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                if (!DW && HALF && tgt >= 0) {
                    const int64_t m = mt + i * 16 + (lane >> 4) * 4;
                    float wv[4];
                    load_some<4>(wt + m, a.M - m, wv);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] += lv * wv[v];
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = tgt >= 0 ? acc[i][j][v] * inv : 0.f;
            }
            if constexpr (HALF) {
                const int64_t m8 = mt + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
#pragma unroll
                for (int i = 0; i < C::FM; i += 2) {
                    const uint4 q = pair_blocks<T>(acc[i][j], acc[i + 1][j]);
                    store_some_raw(o + m8 + i * 16, a.M - m8 - i * 16, __builtin_bit_cast(Raw<T, 8>, q));
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::FM; ++i) {
                    const int64_t m = mt + i * 16 + (lane >> 4) * 4;
                    const float q[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    store_some<4>(o + m, a.M - m, q);
                }
            }
        }
    }
}

template <typename T, typename C, bool DW>
__global__ __launch_bounds__(C::threads, C::per_simd) void xent_product_kernel(const ProductArgs a, int tiles_m,
                                                                               int tiles_n)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    product_tiles<T, C, DW>(a, tiles_m, tiles_n, blockIdx.x, gridDim.x, smem);
}

// dx and dw of a small step in one launch, a workgroup per tile: neither fills the
// chip and both need only G
template <typename T, typename C>
__global__ __launch_bounds__(C::threads, C::per_simd) void xent_both_kernel(const ProductArgs dx, const ProductArgs dw,
                                                                            int dx_m, int dx_n, int dw_m, int dw_n)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int n = dx_m * dx_n * dx.split, b = blockIdx.x;
    if (b < n)
        product_tiles<T, C, false>(dx, dx_m, dx_n, b, n, smem);
    else
        product_tiles<T, C, true>(dw, dw_m, dw_n, b - n, dw_m * dw_n * dw.split, smem);
}

// The slabs of [n][M] added in a fixed order, for dx with the rounding residual:
// a workgroup takes 256 / Q chunks of 4 outputs, Q threads a chunk, thread q slabs
// q, q + Q, .. (few outputs and many slabs would leave most of the chip idle)
template <typename T, bool DW, int Q>
__device__ __forceinline__ void join_slabs(const ProductArgs &a, int block, int blocks, float4 *sum)
{
    constexpr int CH = 256 / Q;
    const int64_t chunks = (a.M + 3) / 4, total = a.n * chunks;
    const float inv = a.scale ? a.scale[1] : 1.f;
    const int k = threadIdx.x % CH, q = threadIdx.x / CH;
    for (int64_t i0 = int64_t(block) * CH; i0 < total; i0 += int64_t(blocks) * CH) {
        const int64_t i = min(i0 + k, total - 1);
        const int64_t row = i / chunks, m = (i - row * chunks) * 4, left = a.M - m;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        const float *src = a.slab + row * a.M + m;
        const int64_t step = a.n * a.M;
        if (left >= 4) {
#pragma unroll 4
            for (int p = q; p < a.split; p += Q) {
                float g[4];
                load_vec<4>(src + p * step, g);
#pragma unroll
                for (int v = 0; v < 4; ++v) f[v] += g[v];
            }
        } else {
            for (int p = q; p < a.split; p += Q)
                for (int v = 0; v < left; ++v) f[v] += src[p * step + v];
        }
        if constexpr (Q > 1) {
            __syncthreads();
            sum[threadIdx.x] = float4{f[0], f[1], f[2], f[3]};
            __syncthreads();
            if (q > 0) continue;
#pragma unroll
            for (int p = 1; p < Q; ++p) {
                const float4 g = sum[p * CH + k];
                f[0] += g.x;
                f[1] += g.y;
                f[2] += g.z;
                f[3] += g.w;
            }
        }
        if (i0 + k >= total) continue;
        int t = 0;
        if constexpr (!DW) {
            t = a.t32[row];
            if (sizeof(T) == 2 && t >= 0) {
                const float lv = static_cast<float>(static_cast<const T *>(a.low)[row]);
                float wv[4];
                load_some<4>(reinterpret_cast<const T *>(static_cast<const char *>(a.w) + t * a.ldw) + m, left, wv);
#pragma unroll
                for (int v = 0; v < 4; ++v) f[v] += lv * wv[v];
            }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = t >= 0 ? f[v] * inv : 0.f;
        store_some<4>(static_cast<T *>(a.out) + row * a.M + m, left, f);
    }
}

template <typename T, int Q>
__global__ __launch_bounds__(256) void xent_join_slabs_kernel(const ProductArgs dx, const ProductArgs dw, int dx_blocks)
{
    __shared__ float4 sum[Q > 1 ? 256 : 1];
    const int b = blockIdx.x;
    if (b < dx_blocks)
        join_slabs<T, false, Q>(dx, b, dx_blocks, sum);
    else
        join_slabs<T, true, Q>(dw, b - dx_blocks, gridDim.x - dx_blocks, sum);
}

template <typename T, typename C, bool DW>
hipError_t launch_tiles(const ProductArgs &a, hipStream_t s)
{
    constexpr bool ONE = DW && sizeof(T) == 2 && C::FM == 8;    // a workgroup for every tile
    const auto kernel = xent_product_kernel<T, C, DW>;
    const int64_t tm = (a.M + C::BM - 1) / C::BM, tn = (a.n + C::BN - 1) / C::BN, all = tm * tn * a.split;
    if (all > (ONE ? max_groups(C::threads) : kMaxTiles)) return hipErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), C::lds_bytes, allowed);
    if (e != hipSuccess) return e;
    const int64_t stages = (a.K * int64_t(sizeof(T)) + 127) / 128 / a.split;
    const int64_t grid = ONE ? all : grid_of<C>(all, stages);
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(C::threads), C::lds_bytes, s, a, int(tm), int(tn));
    return hipGetLastError();
}

template <typename T, bool DW>
hipError_t launch_product(const ProductArgs &a, int tile, hipStream_t s)
{
    switch (tile) {
    case kTile256: return launch_tiles<T, C256, DW>(a, s);
    case kTile128: return launch_tiles<T, C128, DW>(a, s);
    default: return launch_tiles<T, C64, DW>(a, s);
    }
}

template <typename F>
hipError_t with_type(int dtype, F f)
{
    if (dtype == 0) return f(float{});
    if (dtype == 1) return f(_Float16{});
    return f(__bf16{});
}

}  // namespace

hipError_t launch_xent_dx(const ProductArgs &a, int dtype, int tile, hipStream_t s)
{
    return with_type(dtype, [&](auto t) { return launch_product<decltype(t), false>(a, tile, s); });
}

hipError_t launch_xent_dw(const ProductArgs &a, int dtype, int tile, hipStream_t s)
{
    return with_type(dtype, [&](auto t) { return launch_product<decltype(t), true>(a, tile, s); });
}

hipError_t launch_xent_both(const ProductArgs &dx, const ProductArgs &dw, int dtype, hipStream_t s)
{
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        using C = C64;
        const auto kernel = xent_both_kernel<T, C>;
        const int64_t xm = (dx.M + C::BM - 1) / C::BM, xn = (dx.n + C::BN - 1) / C::BN;
        const int64_t wm = (dw.M + C::BM - 1) / C::BM, wn = (dw.n + C::BN - 1) / C::BN;
        const int64_t grid = xm * xn * dx.split + wm * wn * dw.split;
        if (grid > max_groups(C::threads)) return hipErrorInvalidValue;
        static std::atomic<uint64_t> allowed{0};
        const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), C::lds_bytes, allowed);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kernel, dim3(unsigned(grid)), dim3(C::threads), C::lds_bytes, s, dx, dw, int(xm), int(xn),
                           int(wm), int(wn));
        return hipGetLastError();
    });
}

// 16 threads a chunk for 8 slabs and more of fewer than 65536 chunks: 69 rows, 64798
// classes, 256 features, bf16, dx in 64 slabs: step 76.7 us with a thread a chunk, 72.2 so; 64
// rows, 30000 classes, 1024 features, fp16, 16384 chunks 82.0 and 80.9. With few slabs or many
// chunks a thread a chunk fills the chip as well: 300 rows, 40000 classes, 1024 features,
// bf16, 76800 chunks, 199.0 so and 201.1 with 16. (In between it costs 1 us: 300 rows, 5000
// classes, 512 features, fp32 86.3 and 87.5.)
hipError_t launch_xent_join(const ProductArgs *dx, const ProductArgs *dw, int dtype, hipStream_t s)
{
    int64_t blocks[2] = {0, 0}, most = 0;
    bool few = true;
    const ProductArgs *all[2] = {dx, dw};
    for (int k = 0; k < 2; ++k)
        if (all[k]) {
            blocks[k] = all[k]->n * ((all[k]->M + 3) / 4);      // chunks of 4 outputs
            most = std::max(most, blocks[k]);
            few = few && all[k]->split >= 8;
        }
    few = few && most < 65536;
    for (int64_t &b : blocks) b = std::min<int64_t>(few ? (b + 15) / 16 : (b + 255) / 256, 8192);
    return with_type(dtype, [&](auto t) {
        using T = decltype(t);
        const ProductArgs none{}, &x = dx ? *dx : none, &w = dw ? *dw : none;
        const dim3 grid(unsigned(blocks[0] + blocks[1]));
        if (few)
            hipLaunchKernelGGL((xent_join_slabs_kernel<T, 16>), grid, dim3(256), 0, s, x, w, int(blocks[0]));
        else
            hipLaunchKernelGGL((xent_join_slabs_kernel<T, 1>), grid, dim3(256), 0, s, x, w, int(blocks[0]));
        return hipGetLastError();
    });
}

}  // namespace im2win
