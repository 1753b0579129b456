// The feed-forward block's products with an epilogue of their own, the hidden
// features along m:
//   gate   a[n][f] = sum_d Wg[f][d] x[n][d] and u likewise in one tile: its rows
//          alternate, 16 of Wg and the same 16 of Wu, so that a lane holds a and u of
//          the same (n, f); h = act(a) u leaves once, and for the backward pass the
//          factors of dh in du and da, act(a) and u act'(a), in fp32
//   back   dh[n][f] = sum_o Wd[o][f] dy[n][o]; da = dh u act'(a), du = dh act(a)
// The factors are kept rather than formed again: forming them costs a third more products
// in the backward pass, keeping them 8 bytes per (n, f) written and read once; in
// half precision bits they would cost the gradients theirs (half as much error again
// as the outputs' own rounding).
// Bound by the matrix cores where D and O are long, and by the factors' traffic, at which
// all workgroups are at once: 8192 rows, 4096 inputs and outputs, 16384 hidden features,
// bf16: gate 1750 us (1257 TFLOP/s; 1.3 GB written in a sixth of it), back 1120 (982; 1.6 GB
// in a third of it). Workgroups that start apart, so that some are in products while others
// are in epilogues, gain 4 % of back and nothing of gate.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ff_common.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

// rows of two matrices, alternating 16 by 16: row r of the tile is row
// 16 (r / 32) + r % 16 of matrix r / 16 % 2
struct DualOperand {
    const void *p[2];
    int64_t ld[2];           // bytes
    int64_t count;           // rows of each
    int64_t k_end;
};

template <typename T, int TB, int WAVES>
struct DualLoad {
    static constexpr int E = 16 / int(sizeof(T)), KI = 128 / int(sizeof(T));
    static constexpr int blocks = TB / 8, per_wave = blocks / WAVES;
    static_assert(blocks % WAVES == 0 && WAVES % 4 == 0, "a wave's blocks are of one matrix");

    const char *base;        // of this wave's matrix
    uint32_t off[per_wave];

    static __device__ __forceinline__ int block(int wave, int i) { return wave + WAVES * i; }

    __device__ __forceinline__ void init(const DualOperand &op, int64_t first, int wave, int lane)
    {
        const int half = (wave >> 1) & 1;
        const int64_t ld = half ? op.ld[1] : op.ld[0];
        first = first < op.count ? first : op.count - 1;
        const int n = int(op.count - first < TB / 2 ? op.count - first : TB / 2);
        base = static_cast<const char *>(half ? op.p[1] : op.p[0]) + first * ld;
#pragma unroll
        for (int i = 0; i < per_wave; ++i) {
            const int r = block(wave, i) * 8 + (lane >> 3), f = min((r >> 5) * 16 + (r & 15), n - 1);
            off[i] = uint32_t(f) * uint32_t(ld) + (((lane & 7) ^ (lane >> 3)) << 4);
        }
    }
    __device__ __forceinline__ void issue(int64_t s, int i, uint32_t lds, int wave) const
    {
        copy_to_lds_at(base + s * 128, off[i], __builtin_amdgcn_readfirstlane(lds + block(wave, i) * 1024));
    }
    // the last stage of a K that ends inside it: zeros past it
    __device__ __forceinline__ void issue_tail(int64_t stage, int left, uint32_t lds, int wave, int lane) const
    {
        const char *b = base + stage * 128;
#pragma unroll
        for (int i = 0; i < per_wave; ++i) {
            const bool ok = ((lane & 7) ^ (lane >> 3)) * E < left;
            const char *src = ok ? b + off[i] : reinterpret_cast<const char *>(&zero_granule);
            copy_to_lds(src, __builtin_amdgcn_readfirstlane(lds + block(wave, i) * 1024));
        }
    }
};

// 4 consecutive values of each of NB blocks of 16 (16 b + 4 (lane / 16) ..) at p, of
// which `left` are in the row, whole vectors; half precision pairs of blocks as 16-byte
// stores
template <typename T, int NB>
__device__ __forceinline__ void store_blocks(T *p, int left, int lane, const floatx4_t (&v)[NB])
{
    if constexpr (sizeof(T) == 2 && NB % 2 == 0) {
        const int m8 = ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
            const uint4 q = pair_blocks<T>(v[b], v[b + 1]);
            if (m8 + b * 16 < left) store_raw(p + m8 + b * 16, __builtin_bit_cast(Raw<T, 8>, q));
        }
    } else {
        const int m4 = (lane >> 4) * 4;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float q[4] = {v[b][0], v[b][1], v[b][2], v[b][3]};
            if (m4 + b * 16 < left) store_vec<4>(p + m4 + b * 16, q);
        }
    }
}

template <typename T, typename C, bool SAVE>
__global__ __launch_bounds__(C::threads, C::per_simd) void ff_gate_kernel(const FfGate a, int tiles_m, int tiles_n)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    constexpr int NB = C::FM / 2;              // blocks of 16 hidden features of a wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % C::WM, wn = wave / C::WM;
    const int tiles = tiles_m * tiles_n, stages = int((a.Dp + 128 / int(sizeof(T)) - 1) / (128 / int(sizeof(T))));
    const DualOperand A{{a.wg, a.wu}, {a.ldg, a.ldu}, a.F, a.Dp};
    const GemmOperand B{a.x, a.ldx, a.N, a.Dp};
    TilePipe<T, C, false, false, DualLoad<T, C::BM, C::waves>> pipe(smem);
    int64_t f0 = 0, n0 = 0;
    auto start = [&](int t) {
        int tm, tn;
        strip_tile(t, tiles_m, tiles_n, tm, tn);
        f0 = int64_t(tm) * (C::BM / 2);
        n0 = int64_t(tn) * C::BN;
        pipe.start(A, B, f0, n0, 0, stages);
    };
    start(blockIdx.x);
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t ft = f0 + wm * (C::BM / C::WM / 2), nt = n0 + wn * (C::BN / C::WN);
        floatx4_t acc[C::FM][C::FN];
        NoExtra none;
        pipe.template run<0>(false, acc, none);
        if (t + int(gridDim.x) < tiles) start(t + gridDim.x);
        // past the last row and feature h and the factors are zeros: the other passes
        // multiply them
        const bool edge = nt + C::BN / C::WN > a.N || ft + C::BM / C::WM / 2 > a.F;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            if (nt + 16 * j >= a.rows_pad) continue;
            const int64_t row = nt + 16 * j + (lane & 15);
            floatx4_t h[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float g, dg;
                    activate<sizeof(T) == 4>(a.act, acc[2 * b][j][v], g, dg);
                    h[b][v] = g * acc[2 * b + 1][j][v];
                    acc[2 * b][j][v] = g;
                    acc[2 * b + 1][j][v] *= dg;
                }
            if (edge) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (row >= a.N || b * 16 + (lane >> 4) * 4 + v >= a.F - ft)
                            h[b][v] = acc[2 * b][j][v] = acc[2 * b + 1][j][v] = 0.f;
            }
            if constexpr (SAVE) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    if (ft + b * 16 < a.F) {
                        floatx4_t *p = reinterpret_cast<floatx4_t *>(a.to.pre) +
                                       ((nt / 16 + j) * a.to.fblocks + ft / 16 + b) * 128 + lane;
                        p[0] = acc[2 * b][j];
                        p[64] = acc[2 * b + 1][j];
                    }
            }
            store_blocks<T, NB>(static_cast<T *>(a.to.h) + row * a.to.ldh + ft, int(a.Fp - ft), lane, h);
        }
    }
}

// x as the weights' gradients of fp16 read it (ff_common.hpp), a row to a wave
template <typename T>
__device__ __forceinline__ void scale_x(const FfBack &a, int block, int blocks, int waves)
{
    constexpr int E = 16 / int(sizeof(T));
    const int lane = threadIdx.x & 63;
    const float least = dy_scale(a.amax), to = x_scale(a.amax);
    for (int64_t row = int64_t(block) * waves + (threadIdx.x >> 6); row < a.N; row += int64_t(blocks) * waves) {
        const float by = to * fminf(least / a.scale[row], 1.f);
        const T *src = static_cast<const T *>(a.x) + row * a.ldx;
        T *dst = static_cast<T *>(a.to_x) + row * a.ldt;
#pragma unroll 4
        for (int64_t c = lane * E; c < a.Dp; c += 64 * E) {
            float f[E];
            load_some<E>(src + c, a.D - c, f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] *= by;
            store_vec<E>(dst + c, f);
        }
    }
}

// `groups` workgroups for the tiles; fp16: the others for x, where the tiles leave time
template <typename T, typename C>
__global__ __launch_bounds__(C::threads, C::per_simd) void ff_back_kernel(const FfBack a, int tiles_m, int tiles_n,
                                                                          int groups)
{
    constexpr bool SCALED = std::is_same<T, _Float16>::value;
    if constexpr (SCALED)
        if (int(blockIdx.x) >= groups) {
            scale_x<T>(a, int(blockIdx.x) - groups, int(gridDim.x) - groups, C::threads / 64);
            return;
        }
    using E = typename EpiOf<C>::type;         // how the waves hold a tile's sums
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % E::WM, wn = wave / E::WM;
    const int tiles = tiles_m * tiles_n, stages = int((a.O + 128 / int(sizeof(T)) - 1) / (128 / int(sizeof(T))));
    const GemmOperand A{a.wd, a.ldd, a.Fp, a.O};
    const GemmOperand B{a.dy, a.lddy, a.N, a.Op};
    TilePipe<T, C, true, false> pipe(smem);
    int64_t m0 = 0, n0 = 0;
    auto start = [&](int t) {
        int tm, tn;
        strip_tile(t, tiles_m, tiles_n, tm, tn);
        m0 = int64_t(tm) * C::BM;
        n0 = int64_t(tn) * C::BN;
        if constexpr (kSplitWaves<C>)
            pipe.start(A, B, m0, n0, stages * wave / C::groups, stages * (wave + 1) / C::groups);
        else
            pipe.start(A, B, m0, n0, 0, stages);
    };
    start(blockIdx.x);
    for (int t = blockIdx.x; t < tiles; t += groups) {
        const int64_t ft = m0 + wm * (E::BM / E::WM), nt = n0 + wn * (E::BN / E::WN);
        floatx4_t acc[E::FM][E::FN];
        NoExtra none;
        if constexpr (kSplitWaves<C>) {
            floatx4_t part[C::FM][C::FN];
            pipe.template run<0>(false, part, none);
            join_waves<C>(smem, part, acc);
        } else {
            pipe.template run<0>(false, acc, none);
        }
        if (t + groups < tiles) start(t + groups);
        // The factors of H blocks at a time, AHEAD groups of them requested before they are
        // used: one pair at a time, waited for, this epilogue took longer than its products
        // (8192 rows, 4096 outputs, 16384 hidden features, bf16: 1606 us). Past the last
        // row and feature the factors are zeros.
        constexpr int H = E::FM < 2 ? 1 : 2, GROUPS = E::FM / H * E::FN, AHEAD = 2;
        floatx4_t ring[AHEAD + 1][H][2];
        const char *pre = reinterpret_cast<const char *>(a.from.pre) +
                          ((nt / 16) * a.from.fblocks + ft / 16) * 2048;
        auto request = [&](int q) {
            const char *p = pre + (int64_t(q * H / E::FM) * a.from.fblocks + q * H % E::FM) * 2048;
#pragma unroll
            for (int i = 0; i < 2 * H; ++i)
                ring[q % (AHEAD + 1)][i / 2][i % 2] = *reinterpret_cast<const floatx4_t *>(p + i * 1024 + lane * 16);
        };
        float rows[SCALED ? E::FN : 1];        // the rows' own scales
        if constexpr (SCALED)
#pragma unroll
            for (int j = 0; j < E::FN; ++j) rows[j] = a.scale[min(nt + 16 * j + (lane & 15), a.N - 1)];
#pragma unroll
        for (int q = 0; q < AHEAD && q < GROUPS; ++q) request(q);
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
            const int j = q * H / E::FM, i0 = q * H % E::FM;
            const int64_t row = nt + 16 * j + (lane & 15);
            if (q + AHEAD < GROUPS) request(q + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
            floatx4_t da[H], du[H];
#pragma unroll
            for (int i = 0; i < H; ++i) {
                du[i] = acc[i0 + i][j] * ring[q % (AHEAD + 1)][i][0];
                da[i] = acc[i0 + i][j] * ring[q % (AHEAD + 1)][i][1];
            }
            if (nt + 16 * j >= a.rows_pad) continue;
            // past the last row and feature zeros, also beside an infinite dy
            if (nt + 16 * j + 16 > a.N || ft + (i0 + H) * 16 > a.F)
#pragma unroll
                for (int i = 0; i < H; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (row >= a.N || ft + (i0 + i) * 16 + (lane >> 4) * 4 + v >= a.F) da[i][v] = du[i][v] = 0.f;
            if constexpr (SCALED)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    da[i] *= rows[j];
                    du[i] *= rows[j];
                }
            T *g = static_cast<T *>(a.g) + row * 2 * a.from.ldh + ft + i0 * 16;
            store_blocks<T, H>(g, int(a.Fp - ft) - i0 * 16, lane, da);
            store_blocks<T, H>(g + a.from.ldh, int(a.Fp - ft) - i0 * 16, lane, du);
        }
    }
}

template <typename C, typename K, typename A>
hipError_t launch_tiles(K kernel, const A &a, int64_t tm, int64_t tn, int64_t stages, std::atomic<uint64_t> &allowed,
                        hipStream_t s)
{
    if (tm * tn > kMaxTiles) return hipErrorInvalidValue;
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), C::lds_bytes, allowed);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(unsigned(grid_of<C>(tm * tn, stages))), dim3(C::threads), C::lds_bytes, s, a,
                       int(tm), int(tn));
    return hipGetLastError();
}

template <typename T, typename C>
hipError_t launch_gate(const FfGate &a, hipStream_t s)
{
    const int64_t tm = ceil_div(a.Fp, C::BM / 2), tn = ceil_div(a.rows_pad, C::BN);
    const int64_t stages = ceil_div(a.Dp * int64_t(sizeof(T)), 128);
    static std::atomic<uint64_t> allowed[2];
    if (a.to.pre) return launch_tiles<C>(ff_gate_kernel<T, C, true>, a, tm, tn, stages, allowed[1], s);
    return launch_tiles<C>(ff_gate_kernel<T, C, false>, a, tm, tn, stages, allowed[0], s);
}

template <typename T, typename C>
hipError_t launch_back(const FfBack &a, hipStream_t s)
{
    const int64_t tm = ceil_div(a.Fp, C::BM), tn = ceil_div(a.rows_pad, C::BN);
    if (tm * tn > kMaxTiles) return hipErrorInvalidValue;
    static std::atomic<uint64_t> allowed;
    const auto kernel = ff_back_kernel<T, C>;
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kernel), C::lds_bytes, allowed);
    if (e != hipSuccess) return e;
    const int64_t more = std::is_same<T, _Float16>::value ? std::min<int64_t>(ceil_div(a.N, C::threads / 64), 1024) : 0;
    const int64_t groups = std::min(grid_of<C>(tm * tn, ceil_div(a.O * int64_t(sizeof(T)), 128)), max_groups(C::threads) - more);
    hipLaunchKernelGGL(kernel, dim3(unsigned(groups + more)), dim3(C::threads), C::lds_bytes, s, a, int(tm), int(tn),
                       int(groups));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ff_gate(const FfGate &a, int dtype, int tile, hipStream_t s)
{
    return with_ff_type(dtype, [&](auto t) {
        using T = decltype(t);
        switch (tile) {
        case kTile256: return launch_gate<T, C256>(a, s);
        case kTile128: return launch_gate<T, C128>(a, s);
        case kTile64x32: return launch_gate<T, C64x32>(a, s);
        default: return launch_gate<T, C64>(a, s);
        }
    });
}

hipError_t launch_ff_back(const FfBack &a, int dtype, int tile, hipStream_t s)
{
    return with_ff_type(dtype, [&](auto t) {
        using T = decltype(t);
        switch (tile) {
        case kTile256: return launch_back<T, C256>(a, s);
        case kTile128: return launch_back<T, C128>(a, s);
        case kTile32K:
            // (a tile of 32 columns in half precision has too few granules for the
            // transposed reads)
            if constexpr (sizeof(T) == 4) return launch_back<T, C32K>(a, s);
            return hipErrorInvalidValue;
        default: return launch_back<T, C64>(a, s);
        }
    });
}

}  // namespace im2win
