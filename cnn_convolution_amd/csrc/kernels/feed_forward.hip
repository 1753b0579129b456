// Gated feed-forward block (im2win_block.h): the plan, the small kernels, the kernels
// for few rows, and the sequence of launches.
//
// Forward: the gate launch (ff_tiles.hip) forms both projections, the activation and
// the product and leaves h; a plain product (ff_products.hip) leaves y. Backward: the
// back launch leaves da and du from dy, Wd and the saved factors, in fp16 x too as the weights'
// gradients read it; then dx, dWd and dWg with dWu.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ff_common.hpp"
#include "head_gemm.hpp"
#include "head_vec.hpp"

namespace im2win {
namespace {

// ---- rows padded to whole granules, the rows' largest |dy| --------------------------

struct PadJob {
    const void *src;
    void *dst;
    int64_t ld, rows, D, Dp; // elements; dst: rows of Dp, ldd apart
    int64_t ldd;
    int64_t end;             // workgroups up to and with this job's
};
struct PadArgs {
    PadJob job[5];
    int count;
    const void *dy;          // of which the largest finite |values| are wanted, or null
    const void *x;           // and its, of rows whose dy is not 0
    int64_t lddy, ldx, N, O, D;
    float *amax;             // [2][kAmaxParts]: of a workgroup's rows, of dy and of x
    float *scale;            // [N]: S of each row
};

template <typename T>
__global__ __launch_bounds__(256) void ff_pad_kernel(const PadArgs a)
{
    constexpr int E = 16 / int(sizeof(T));
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t copies = a.count ? a.job[a.count - 1].end : 0;
    int64_t b = blockIdx.x;
    if (b >= copies) {
        // a row to a wave, or where there are few to a workgroup
        __shared__ float red[3][4];
        const bool few = a.N <= kAmaxParts;
        const int lanes = few ? 256 : 64, at = few ? int(threadIdx.x) : lane;
        b -= copies;
        float most = 0.f, most_x = 0.f, own = 0.f;
        bool some = false;
        // the largest finite |value| of a row that these lanes read, and whether it has any but
        // 0, by the bits of two fp16 values at a time (as floats, one load after the other, 4097
        // rows of 1032 took 20 us for 12)
        typedef uint16_t half2_t __attribute__((ext_vector_type(2)));
        const auto row_max = [&](const void *p, int64_t ld, int64_t r, int64_t n, bool &any) {
            const uint16_t *row = static_cast<const uint16_t *>(p) + r * ld;
            half2_t m = {0, 0};
            uint32_t seen = 0;
            const auto take = [&](uint32_t d) {
                d &= 0x7FFF7FFFu;
                seen |= d;
                // (from 0x7C00 on: infinite or NaN)
                const uint32_t no = (d + 0x04000400u) & 0x80008000u;
                m = __builtin_elementwise_max(m, __builtin_bit_cast(half2_t, d & ~(no | (no - (no >> 15)))));
            };
            if (n < E) {
                if (at < n) take(row[at]);
            } else {
                // past the end the last ones again
                for (int64_t c = at * E; c - at * E < n; c += 4 * lanes * E) {
                    Raw<uint16_t, E> q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = load_raw<uint16_t, E>(row + min(c + i * lanes * E, n - E));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < E / 2; ++e) take(q[i].d[e]);
                }
            }
            any = __any(seen != 0);
            float f = float(__builtin_bit_cast(_Float16, uint16_t(max(m[0], m[1]))));
            for (int k = 1; k < 64; k <<= 1) f = fmaxf(f, __shfl_xor(f, k, 64));
            return f;
        };
        for (int64_t r = few ? b : b * 4 + wave; r < a.N; r += few ? kAmaxParts : 4 * kAmaxParts) {
            bool any = false, any_x = false;
            own = row_max(a.dy, a.lddy, r, a.O, any);
            const float x = row_max(a.x, a.ldx, r, a.D, any_x);
            some = any;
            most = fmaxf(most, own);
            if (any || few) most_x = fmaxf(most_x, x);
            if (!few && lane == 0) a.scale[r] = any ? scale_of(own) : kZeroRow;
        }
        if (lane == 0) {
            red[0][wave] = most;
            red[1][wave] = most_x;
            red[2][wave] = some ? 1.f : 0.f;
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            const auto of = [&](const float (&v)[4]) { return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])); };
            const float m = of(red[0]);
            const bool zeros = few && of(red[2]) == 0.f;      // the workgroup's one row, or none
            a.amax[b] = m;
            a.amax[kAmaxParts + b] = zeros ? 0.f : of(red[1]);
            if (few && b < a.N) a.scale[b] = zeros ? kZeroRow : scale_of(m);
        }
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
        store_vec<E>(static_cast<T *>(j.dst) + row * j.ldd + c, f);
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
// At most FF_ROWS rows, NB blocks of 16: the weights are read once and that read is all
// that counts. A workgroup takes 16 rows of a weight matrix (of Wg and of Wu for h), its
// waves split K; the weights go from memory straight to the lanes that multiply them (16
// rows x 64 bytes a load, the matrix cores' own layout, so no LDS and no barrier until the
// waves' sums are joined, no padded copies of odd rows), x or h come from the caches.
// Rows past N repeat the last one. In half precision h is kept in two parts, rounded and
// what that took: its rounding would be as large in y as y's own.
// 1 row, 4096 inputs and outputs, 8192 hidden features, bf16: h 23.3 us (5.8 TB/s), y
// 15.5 (4.3). 37 rows, 1001, 2003, fp16: h 11.9 us, y 8.3, the latency of a few loads one
// after the other. Above 16 rows tiles are faster where they can read in place (2048, 8192,
// bf16: 24 rows 28 us, 16 rows here 33), but their y has 1.4 times the error.

// A row of K values. ODD: half-precision rows that start at any element are read as the
// dwords that hold them and shifted into place, for 16-byte loads that start between
// dwords take twice the time (16 rows, 1001 inputs, 2000 hidden features, fp16: h 10.1 us,
// 8.3 so, 1002 inputs 6.5). No dword is touched that holds nothing of the vector.
template <typename T, bool ODD>
struct Row {
    static constexpr int E = 16 / int(sizeof(T));
    const T *row;
    uint32_t shift;          // bits

    __device__ __forceinline__ void init(const T *p)
    {
        row = p;
        shift = ODD ? uint32_t(reinterpret_cast<uintptr_t>(p) & 2) * 8 : 0;
    }
    // E values from `k` on, all in the row
    __device__ __forceinline__ uint4 vec(int64_t k) const
    {
        if constexpr (!ODD) {
            const Raw<T, E> r = load_raw<T, E>(row + k);
            return uint4{r.d[0], r.d[1], r.d[2], r.d[3]};
        } else {
            typedef uint32_t vec4 __attribute__((ext_vector_type(4), aligned(4)));
            const char *p = reinterpret_cast<const char *>(row + k) - shift / 8;
            const vec4 d = *reinterpret_cast<const vec4 *>(p);
            const uint32_t e = *reinterpret_cast<const uint32_t *>(p + (shift ? 16 : 12));
            return uint4{__builtin_amdgcn_alignbit(d[1], d[0], shift), __builtin_amdgcn_alignbit(d[2], d[1], shift),
                         __builtin_amdgcn_alignbit(d[3], d[2], shift), __builtin_amdgcn_alignbit(e, d[3], shift)};
        }
    }
    // up to the row's end and zeros past it, without a branch (element by element, each
    // a wait behind a branch, the step that K ends in took longer than all others)
    __device__ __forceinline__ uint4 end(int64_t k, int64_t K) const
    {
        if (K >= E) {
            const Raw<T, E> r = load_row<T, E, false>(row, k, K);
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
};

template <typename T>
constexpr int kFragK = 64 / int(sizeof(T));    // K of a fragment pair: 16 bytes a lane

// The waves' sums of M sets of NB blocks, added in order: wave w < NB is left with block
// w of each set.
template <int WAVES, int M, int NB>
__device__ __forceinline__ void join_parts(const floatx4_t (&acc)[M][NB], floatx4_t (&out)[M], floatx4_t *part)
{
    static_assert(NB <= WAVES, "a wave per block");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) part[((wave * M + m) * NB + b) * 64 + lane] = acc[m][b];
    __syncthreads();
    if (wave >= NB) return;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        out[m] = part[(m * NB + wave) * 64 + lane];
        for (int w = 1; w < WAVES; ++w) out[m] += part[((w * M + m) * NB + wave) * 64 + lane];
    }
}

template <typename T, int WAVES, int NB, bool SAVE, bool ODD>
__global__ __launch_bounds__(WAVES * 64) void ff_rows_gate_kernel(const FfRows a)
{
    constexpr int KF = kFragK<T>, U = 4;       // fragments in flight per matrix
    __shared__ floatx4_t part[WAVES * 2 * NB * 64];
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < a.counts; i += WAVES * 64) a.count[i] = 0;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t f0 = int64_t(blockIdx.x) * 16, f = min(f0 + (lane & 15), a.F - 1);
    Row<T, ODD> wg, wu, x[NB];
    wg.init(static_cast<const T *>(a.wg) + f * a.ldg);
    wu.init(static_cast<const T *>(a.wu) + f * a.ldu);
#pragma unroll
    for (int b = 0; b < NB; ++b)
        x[b].init(static_cast<const T *>(a.x) + min(int64_t((blockIdx.y * NB + b) * 16 + (lane & 15)), a.N - 1) * a.ldx);
    const int q = (lane >> 4) * (16 / int(sizeof(T)));
    const int64_t steps = (a.D + KF - 1) / KF, whole = a.D / KF;
    int64_t s = steps * wave / WAVES;
    const int64_t end = steps * (wave + 1) / WAVES;
    floatx4_t acc[2][NB] = {};
    // the step that K ends in, by the wave that has it: its loads go out first
    uint4 tg{}, tu{}, tx[NB] = {};
    const bool tail = end > whole;
    if (tail) {
        tg = wg.end(whole * KF + q, a.D);
        tu = wu.end(whole * KF + q, a.D);
#pragma unroll
        for (int b = 0; b < NB; ++b) tx[b] = x[b].end(whole * KF + q, a.D);
    }
    // the loads of U steps at a time; in the last batch past the wave's last step that
    // one again, unused
    const int64_t last = min(end, whole) - 1;
    auto batch = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        uint4 g[U], u[U], xf[NB][U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t k = (FULL ? s + i : min(s + i, last)) * KF + q;
            g[i] = wg.vec(k);
            u[i] = wu.vec(k);
#pragma unroll
            for (int b = 0; b < NB; ++b) xf[b][i] = x[b].vec(k);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!FULL && s + i > last) break;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                acc[0][b] = mfma_half<T>(g[i], xf[b][i], acc[0][b]);
                acc[1][b] = mfma_half<T>(u[i], xf[b][i], acc[1][b]);
            }
        }
    };
    for (; s + U - 1 <= last; s += U) batch(std::true_type{});
    if (s <= last) batch(std::false_type{});
    if (tail)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            acc[0][b] = mfma_half<T>(tg, tx[b], acc[0][b]);
            acc[1][b] = mfma_half<T>(tu, tx[b], acc[1][b]);
        }
    floatx4_t sum[2];
    join_parts<WAVES, 2, NB>(acc, sum, part);
    // waves past the blocks of rows that there are leave the zeros of those that there are not
    if (wave >= NB && (!SAVE || blockIdx.y > 0)) return;
    const int rb = (wave < NB ? blockIdx.y : gridDim.y - 1) * NB + wave;     // block of rows
    if (rb >= a.blocks) return;
    if (wave >= NB) sum[0] = sum[1] = floatx4_t{};
    const int64_t row = rb * 16 + (lane & 15), m = f0 + (lane >> 4) * 4;
    float h[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const bool in = row < a.N && m + v < a.F;
        float g, dg;
        activate<sizeof(T) == 4>(a.act, sum[0][v], g, dg);
        h[v] = in ? g * sum[1][v] : 0.f;
        sum[0][v] = in ? g : 0.f;
        sum[1][v] = in ? sum[1][v] * dg : 0.f;
    }
    if constexpr (SAVE) {
        floatx4_t *p = reinterpret_cast<floatx4_t *>(a.to.pre) + (rb * a.to.fblocks + blockIdx.x) * 128 + lane;
        p[0] = sum[0];
        p[64] = sum[1];
    }
    if (m >= a.Fp || (!SAVE && row >= a.N)) return;
    const Raw<T, 4> hi = to_raw<T, 4>(h);
    store_raw(static_cast<T *>(a.to.h) + row * a.to.ldh + m, hi);
    if (sizeof(T) == 4 || row >= a.N) return;
    float rest[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)              // (an infinite h has no second part)
        rest[v] = fabsf(element(hi, v)) < __builtin_inff() ? h[v] - element(hi, v) : 0.f;
    store_vec<4>(static_cast<T *>(a.lo) + row * a.to.ldh + m, rest);
}

template <typename T, int WAVES, int NB, bool ODD>
__global__ __launch_bounds__(WAVES * 64) void ff_rows_down_kernel(const FfRows a)
{
    constexpr int KF = kFragK<T>, U = 4;
    constexpr bool HALF = sizeof(T) == 2;
    __shared__ floatx4_t part[WAVES * NB * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t o0 = int64_t(blockIdx.x) * 16, o = min(o0 + (lane & 15), a.O - 1);
    Row<T, ODD> w;
    w.init(static_cast<const T *>(a.wd) + o * a.ldd);
    const int q = (lane >> 4) * (16 / int(sizeof(T)));
    Row<T, false> hi[NB], lo[NB];              // whole vectors up to Fp, zeros past F
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t at = min(int64_t((blockIdx.y * NB + b) * 16 + (lane & 15)), a.N - 1) * a.to.ldh;
        hi[b].init(static_cast<const T *>(a.to.h) + at);
        lo[b].init(static_cast<const T *>(a.lo) + at);
    }
    const int64_t steps = (a.F + KF - 1) / KF, whole = a.F / KF;
    const int turn = blockIdx.z * WAVES + wave, turns = gridDim.z * WAVES;
    int64_t s = steps * turn / turns;
    const int64_t end = steps * (turn + 1) / turns;
    floatx4_t acc[1][NB] = {};
    uint4 tw{}, th[NB] = {}, tl[NB] = {};
    const bool tail = end > whole;
    if (tail) {
        tw = w.end(whole * KF + q, a.F);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            th[b] = hi[b].end(whole * KF + q, a.Fp);
            if (HALF) tl[b] = lo[b].end(whole * KF + q, a.Fp);
        }
    }
    const int64_t last = min(end, whole) - 1;
    auto batch = [&](auto full) {
        constexpr bool FULL = decltype(full)::value;
        uint4 wf[U], hf[NB][U], lf[NB][U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t k = (FULL ? s + i : min(s + i, last)) * KF + q;
            wf[i] = w.vec(k);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                hf[b][i] = hi[b].vec(k);
                if (HALF) lf[b][i] = lo[b].vec(k);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!FULL && s + i > last) break;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                acc[0][b] = mfma_half<T>(wf[i], hf[b][i], acc[0][b]);
                if (HALF) acc[0][b] = mfma_half<T>(wf[i], lf[b][i], acc[0][b]);
            }
        }
    };
    for (; s + U - 1 <= last; s += U) batch(std::true_type{});
    if (s <= last) batch(std::false_type{});
    if (tail)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            acc[0][b] = mfma_half<T>(tw, th[b], acc[0][b]);
            if (HALF) acc[0][b] = mfma_half<T>(tw, tl[b], acc[0][b]);
        }
    floatx4_t sum[1];
    join_parts<WAVES, 1, NB>(acc, sum, part);
    if (gridDim.z > 1) {
        // the workgroup that comes last adds all parts, in their order. Parts pass the L2
        // caches (stores and loads of the device's scope, the count taken once the stores
        // are done): a fence that writes a whole L2 back takes 100 us and more here
        __shared__ int last_one;
        const int64_t tile = blockIdx.y * int64_t(gridDim.x) + blockIdx.x, tiles = int64_t(gridDim.x) * gridDim.y;
        float *slab = a.slab + (tile * NB + wave) * 256 + lane;
        const int64_t part_step = tiles * NB * 256;
        if (wave < NB) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                __hip_atomic_store(slab + blockIdx.z * part_step + v * 64, sum[0][v], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        __syncthreads();
        if (threadIdx.x == 0)
            last_one = __hip_atomic_fetch_add(a.count + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                       int(gridDim.z) - 1;
        __syncthreads();
        if (!last_one || wave >= NB) return;
        sum[0] = floatx4_t{};
        for (unsigned p = 0; p < gridDim.z; ++p)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                sum[0][v] += __hip_atomic_load(slab + p * part_step + v * 64, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const int64_t row = (blockIdx.y * NB + wave) * 16 + (lane & 15), m = o0 + (lane >> 4) * 4;
    if (wave >= NB || row >= a.N) return;
    const float y[4] = {sum[0][0], sum[0][1], sum[0][2], sum[0][3]};
    store_some<4>(static_cast<T *>(a.y) + row * a.ldy + m, a.O - m, y);
}

// workgroups up to which each block of rows has workgroups of its own, which read the same
// weights again (64 rows, fp32, 512 inputs, 1024 hidden features, 256 of them: h 6.8 us,
// 11.8 with 64 rows a workgroup; 2048 inputs, 4096 hidden features, 1024: 79 us in all, 74)
constexpr int64_t kRowsGroups = 512;
// parts of y's K: as many as leave at most a workgroup per CU, for with few outputs each
// workgroup reads all of h and few CUs do (bf16, 16 rows, 1024 outputs, 4096 hidden features:
// 8 us, 13 in one part; fp32, 64 rows, 2048 outputs, 8192: 45 us, 78). Two workgroups a CU
// are slower (bf16, 1 row, 4096 outputs, 8192: 21 us, 14 in one part).
constexpr int64_t kPartGroups = 256, kMaxParts = 16;

// ---- plan ------------------------------------------------------------------------------

struct FfPlan {
    bool few;                // the kernels for few rows
    bool fits;               // no launch has more tiles than one can
    int row_blocks, parts, tiles;   // blocks of rows a workgroup, parts of y's K, workgroups of a part if there are some
    int64_t off_count;
    int64_t Dp, Fp, Op, rows_pad, fblocks;
    int64_t ldd, ldf, ldo;   // strides of rows of D, F and O in the workspace
    bool copy_x, copy_g, copy_u, copy_d, copy_y;   // rows not made of 16-byte granules
    int gate_tile, y_tile, y_split, back_tile, dx_tile, dx_split, dd_tile, dd_split, dg_tile, dg_split;
    int all_tile;            // of dx, dWd, dWg and dWu in one launch, or -1
    int64_t off_x, off_g, off_u, off_d, off_dy, off_h, off_lo, off_slab_x, off_slab_d, off_slab_g, off_grad, off_amax, off_scale, bytes;
    int64_t pre_bytes;       // of saved, before h
};

int64_t take(FfPlan &p, int64_t bytes)
{
    const int64_t at = p.bytes;
    p.bytes += round_up(bytes, 256);
    return at;
}

// tile of a product that is not split (back: of dh, else of the gate)
int pick_tile(int64_t M, int64_t N, int64_t stages, int dtype, int out_bytes, int saved_bytes, bool back)
{
    double best = 1e30;
    int tile = 0;
    for (int t = 0; t < 5; ++t) {
        if (t == kTile32K && (!back || dtype)) continue;
        // W would be read three times and more; Wd's columns take twice the time in tiles
        // of 32 rows (24 rows, 2048 outputs, 8192 hidden features, bf16: 13 us, 21)
        if (t == kTile64x32 && (back || N > 64)) continue;
        const int64_t own = t == kTile32K ? ceil_div(stages, 4) : stages;
        // what is saved or read back goes at the chip's rate, hidden by nothing: all
        // workgroups are in their epilogues at once (4097 x 1032 x 3001, fp16, gate with
        // tiles of 256 95 us, of 128 114; 8192 x 2048 x 8192, bf16, back 363 and 397)
        const double us = product_us(kShapes[t], M, N, own, 1, dtype, out_bytes) +
                          double(M) * double(N) * saved_bytes / 5e6;
        if (us < best * 0.98) {
            best = us;
            tile = t;
        }
    }
    return tile;
}

struct Product {
    int64_t M, N, stages;
    int64_t outs;            // N: rows of each

    int64_t rows(const TileShape &t) const { return outs > 1 ? outs * round_up(N, t.n) : N; }
};

// of a split product's slabs: written, read once more at about 3 TB/s by a launch of
// their own
double slab_us(const Product &q, int split) { return 5.0 + double(split) * double(q.M) * double(q.N * q.outs) * 4 / 3e6; }

// tile and split of a product by itself, and its microseconds
double pick(const Product &q, int dtype, int *tile, int *split)
{
    double best = 1e30;
    for (int t = 0; t < 3; ++t)
        for (int sp : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
            if (sp > 1 && (q.stages / sp < 4 || int64_t(sp) * q.M * q.N * q.outs * 4 > kSlabBytes)) break;
            const double us = product_us(kShapes[t], q.M, q.rows(kShapes[t]), q.stages, sp, dtype, sp > 1 ? 4 : int(elem(dtype))) +
                              (sp > 1 ? slab_us(q, sp) : 0.0);
            if (us < best * 0.98) {
                best = us;
                *tile = t;
                *split = sp;
            }
        }
    return best;
}

// whether a launch takes the product's tiles; one: with a workgroup for each
bool fits(const Product &q, int dtype, int tile, int split, bool columns)
{
    const TileShape &t = kShapes[tile];
    const bool one = columns && dtype && tile == kTile256;
    return ceil_div(q.M, t.m) * ceil_div(q.N, t.n) * q.outs * split <= (one ? max_groups(C256::threads) : kMaxTiles);
}

// microseconds of three products in one launch of tiles t: what the chip's slots have to
// do, but at least the longest workgroup; a product's K is split where its workgroups
// would be longer than that share
double together_us(int t, const Product (&q)[3], int dtype, int (&split)[3])
{
    const TileShape &c = kShapes[t];
    const double stage = (dtype == 0 ? c.f32 : c.half)[c.per_cu - 1], slots = double(kCus * c.per_cu);
    const double fixed = c.fixed + double(c.m * c.n) * 7.0 / 65536;
    double work = 0.0, longest = 0.0, slabs = 0.0;
    for (const Product &p : q)
        work += double(ceil_div(p.M, c.m) * ceil_div(p.rows(c), c.n)) * (stage * double(p.stages) + fixed) / slots;
    for (int k = 0; k < 3; ++k) {
        split[k] = 1;
        while (split[k] < 32 && stage * double(q[k].stages) / split[k] > 1.2 * work + 3.0 &&
               q[k].stages / (2 * split[k]) >= 4 && int64_t(2 * split[k]) * q[k].M * q[k].N * q[k].outs * 4 <= kSlabBytes)
            split[k] *= 2;
        if (split[k] > 1) slabs += slab_us(q[k], split[k]) - 5.0;
        longest = std::max(longest, stage * double(ceil_div(q[k].stages, split[k])) + fixed);
    }
    return std::max(work, longest) + 0.25 * longest + (slabs > 0.0 ? slabs + 5.0 : 0.0);
}

FfPlan plan_common(const FfSizes &z)
{
    FfPlan p{};
    p.fits = true;
    const int64_t es = elem(z.dtype), e = 16 / es;
    p.Dp = round_up(z.D, e);
    p.Fp = round_up(z.F, e);
    p.Op = round_up(z.O, e);
    // whole cache lines: a stage's 128 bytes of a row are one (4097 rows, 1032 inputs, 3000
    // hidden features, fp16, rows of Fp: y 56 us; 8 features more fill their lines: 49)
    p.ldd = round_up(z.D, 128 / es);
    p.ldf = round_up(z.F, 128 / es);
    p.ldo = round_up(z.O, 128 / es);
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
    if (p.copy_x) p.off_x = take(p, z.N * p.ldd * es);
    if (p.copy_g) p.off_g = take(p, z.F * p.ldd * es);
    if (p.copy_u) p.off_u = take(p, z.F * p.ldd * es);
    if (p.copy_d) p.off_d = take(p, z.O * p.ldf * es);
}

FfPlan plan_fwd(const FfSizes &z, bool saved)
{
    FfPlan p = plan_common(z);
    if (z.N == 0) return p;
    const int64_t es = elem(z.dtype), ki = 128 / es;
    p.few = z.N <= 16 || (z.N <= FF_ROWS && (!z.dtype || p.copy_g || p.copy_u || p.copy_d));
    if (p.few) {
        if (!saved) p.off_h = take(p, z.N * p.ldf * es);
        if (z.dtype) p.off_lo = take(p, z.N * p.ldf * es);
        const int64_t nb = ceil_div(z.N, 16);
        p.row_blocks = nb == 1 || ceil_div(z.F, 16) * nb <= kRowsGroups ? 1 : nb == 2 ? 2 : 4;
        const int waves = p.row_blocks == 1 ? 16 : 8;
        const int64_t tiles = ceil_div(z.O, 16) * ceil_div(nb, p.row_blocks), steps = ceil_div(p.Fp * es, 64);
        p.parts = 1;
        while (p.parts < kMaxParts && tiles * p.parts * 2 <= kPartGroups && steps / (p.parts * 2) >= 2 * waves)
            p.parts *= 2;
        if (p.parts > 1) {
            p.off_slab_x = take(p, tiles * p.row_blocks * p.parts * 1024);
            p.off_count = take(p, tiles * 4);
            p.tiles = int(tiles);
        }
        return p;
    }
    plan_copies(p, z);
    if (!saved) p.off_h = take(p, p.rows_pad * p.ldf * es);
    p.gate_tile = pick_tile(2 * p.Fp, z.N, ceil_div(p.Dp, ki), z.dtype, int(es / 2), saved ? 4 : 0, false);
    const Product gate{2 * p.Fp, p.rows_pad, 0, 1}, y{z.O, z.N, ceil_div(p.Fp, ki), 1};
    pick(y, z.dtype, &p.y_tile, &p.y_split);
    p.fits = fits(gate, z.dtype, p.gate_tile, 1, false) && fits(y, z.dtype, p.y_tile, p.y_split, false);
    if (p.y_split > 1) p.off_slab_x = take(p, p.y_split * z.N * z.O * 4);
    return p;
}

FfPlan plan_bwd(const FfSizes &z)
{
    FfPlan p = plan_common(z);
    if (z.N == 0) return p;
    const int64_t es = elem(z.dtype), ki = 128 / es;
    if (z.dtype == 1) p.copy_x = false;        // x is written anew
    plan_copies(p, z);
    if (p.copy_y) p.off_dy = take(p, z.N * p.ldo * es);
    p.off_grad = take(p, p.rows_pad * 2 * p.ldf * es);
    if (z.dtype == 1) {
        p.off_x = take(p, z.N * p.ldd * es);
        p.off_amax = take(p, 2 * kAmaxParts * 4);
        p.off_scale = take(p, z.N * 4);
    }
    p.back_tile = pick_tile(p.Fp, z.N, ceil_div(z.O, ki), z.dtype, 0, int(8 + 2 * es), true);
    const Product dx{z.D, z.N, 2 * ceil_div(z.F, ki), 1}, dd{z.F, z.O, ceil_div(z.N, ki), 1}, dg{z.D, z.F, dd.stages, 2};
    double apart = 0.0;
    apart += pick(dx, z.dtype, &p.dx_tile, &p.dx_split);
    apart += pick(dd, z.dtype, &p.dd_tile, &p.dd_split);
    apart += pick(dg, z.dtype, &p.dg_tile, &p.dg_split);
    p.fits = fits(Product{p.Fp, p.rows_pad, 0, 1}, z.dtype, p.back_tile, 1, false) &&
             fits(dx, z.dtype, p.dx_tile, p.dx_split, false) && fits(dd, z.dtype, p.dd_tile, p.dd_split, true) &&
             fits(dg, z.dtype, p.dg_tile, p.dg_split, true);
    p.all_tile = -1;
    const Product all[3] = {dx, dd, dg};
    for (int t : {kTile128, kTile64}) {
        int split[3];
        const double us = together_us(t, all, z.dtype, split);
        int64_t groups = 0;
        for (int k = 0; k < 3; ++k)
            groups += ceil_div(all[k].M, kShapes[t].m) * ceil_div(all[k].rows(kShapes[t]), kShapes[t].n) * split[k];
        if (us > apart * 0.95 || groups > max_groups(256)) continue;
        apart = us;
        p.all_tile = t;
        p.dx_split = split[0];
        p.dd_split = split[1];
        p.dg_split = split[2];
    }
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
    auto add = [&](bool copy, const void *src, int64_t ld, int64_t rows, int64_t D, int64_t Dp, int64_t ldd,
                   int64_t off, const void *&to, int64_t &to_ld) {
        to = src;
        to_ld = ld * es;
        if (!copy) return;
        to = ws + off;
        to_ld = ldd * es;
        groups += ceil_div(rows, 4);
        pad.job[pad.count++] = PadJob{src, ws + off, ld, rows, D, Dp, ldd, groups};
    };
    add(p.copy_x, a.x, z.ldx, z.N, z.D, p.Dp, p.ldd, p.off_x, r->x, r->ldx);
    add(p.copy_g, a.wg, z.ldg, z.F, z.D, p.Dp, p.ldd, p.off_g, r->wg, r->ldg);
    add(p.copy_u, a.wu, z.ldu, z.F, z.D, p.Dp, p.ldd, p.off_u, r->wu, r->ldu);
    add(p.copy_d, a.wd, z.ldd, z.O, z.F, p.Fp, p.ldf, p.off_d, r->wd, r->ldd);
    if (backward) {
        add(p.copy_y, a.dy, z.ldy, z.N, z.O, p.Op, p.ldo, p.off_dy, r->dy, r->lddy);
        if (z.dtype == 1) {
            pad.dy = a.dy;
            pad.x = a.x;
            pad.lddy = z.ldy;
            pad.ldx = z.ldx;
            pad.D = z.D;
            pad.N = z.N;
            pad.O = z.O;
            pad.amax = reinterpret_cast<float *>(ws + p.off_amax);
            pad.scale = reinterpret_cast<float *>(ws + p.off_scale);
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
    return FfSaved{reinterpret_cast<float *>(c), p.fblocks, c ? c + p.pre_bytes : h, p.ldf};
}

// nb blocks of rows: NB at a time by a workgroup, the others by further workgroups
template <typename T, int NB, bool ODD>
hipError_t launch_rows(const FfRows &a, int64_t nb, int parts, hipStream_t s)
{
    constexpr int GATE = NB == 1 ? 8 : 4, DOWN = NB == 1 ? 16 : 8;
    const dim3 gate(unsigned(ceil_div(a.F, 16)), unsigned(ceil_div(nb, NB)));
    const dim3 down(unsigned(ceil_div(a.O, 16)), gate.y, unsigned(parts));
    if (a.to.pre)
        hipLaunchKernelGGL((ff_rows_gate_kernel<T, GATE, NB, true, ODD>), gate, dim3(GATE * 64), 0, s, a);
    else
        hipLaunchKernelGGL((ff_rows_gate_kernel<T, GATE, NB, false, ODD>), gate, dim3(GATE * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ff_rows_down_kernel<T, DOWN, NB, ODD>), down, dim3(DOWN * 64), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_rows(const FfRows &a, int dtype, int row_blocks, int parts, hipStream_t s)
{
    const int64_t nb = ceil_div(a.N, 16);
    return with_ff_type(dtype, [&](auto t) {
        using T = decltype(t);
        const auto blocks = [&](auto odd) {
            constexpr bool ODD = decltype(odd)::value;
            if (row_blocks == 1) return launch_rows<T, 1, ODD>(a, nb, parts, s);
            if (row_blocks == 2) return launch_rows<T, 2, ODD>(a, nb, parts, s);
            return launch_rows<T, 4, ODD>(a, nb, parts, s);
        };
        if constexpr (sizeof(T) == 2) {
            bool odd = (a.ldx | a.ldg | a.ldu | a.ldd) & 1;
            for (const void *p : {a.x, a.wg, a.wu, a.wd}) odd = odd || reinterpret_cast<uintptr_t>(p) % 4 != 0;
            if (odd) return blocks(std::true_type{});
        }
        return blocks(std::false_type{});
    });
}

}  // namespace

int64_t ff_saved_bytes(const FfSizes &z)
{
    const FfPlan p = plan_common(z);
    return p.pre_bytes + p.rows_pad * p.ldf * elem(z.dtype);
}

int64_t ff_fwd_ws_bytes(const FfSizes &z, bool saved)
{
    const FfPlan p = plan_fwd(z, saved);
    return p.fits ? p.bytes : -1;
}
int64_t ff_bwd_ws_bytes(const FfSizes &z)
{
    const FfPlan p = plan_bwd(z);
    return p.fits ? p.bytes : -1;
}

hipError_t launch_ff_fwd(const FfArgs &a, hipStream_t s)
{
    const FfSizes &z = a.z;
    if (z.N == 0) return hipSuccess;
    const FfPlan p = plan_fwd(z, a.saved != nullptr);
    char *ws = static_cast<char *>(a.ws);
    const int64_t es = elem(z.dtype);
    const FfSaved to = saved_of(p, a.saved, ws + p.off_h);
    if (p.few)
        return launch_rows(FfRows{a.x, a.wg, a.wu, a.wd, z.ldx, z.ldg, z.ldu, z.ldd, z.ldy, z.N, z.D, z.F, z.O, p.Fp, to,
                                  ws + p.off_lo, a.y, z.act, int(ceil_div(a.saved ? p.rows_pad : z.N, 16)),
                                  p.parts > 1 ? reinterpret_cast<float *>(ws + p.off_slab_x) : nullptr,
                                  p.parts > 1 ? reinterpret_cast<int *>(ws + p.off_count) : nullptr, p.tiles},
                           z.dtype, p.row_blocks, p.parts, s);
    FfRead r{};
    hipError_t e = launch_pads(p, a, false, &r, s);
    if (e != hipSuccess) return e;
    const FfGate g{r.x, r.wg, r.wu, r.ldx, r.ldg, r.ldu, z.N, z.F, p.Dp, p.rows_pad, p.Fp, to, z.act};
    if ((e = launch_ff_gate(g, z.dtype, p.gate_tile, s)) != hipSuccess) return e;
    FfProduct y{};
    y.a[0] = r.wd;
    y.lda[0] = r.ldd;
    y.b = to.h;
    y.ldb = p.ldf * es;
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
    const bool scaled = z.dtype == 1;
    const float *amax = scaled ? reinterpret_cast<const float *>(ws + p.off_amax) : nullptr;
    const float *scale = scaled ? reinterpret_cast<const float *>(ws + p.off_scale) : nullptr;
    const FfSaved from = saved_of(p, a.saved, nullptr);
    const FfBack back{r.dy, r.wd, r.lddy, r.ldd, z.N, z.F, z.O, p.Op, p.rows_pad, p.Fp, from, ws + p.off_grad,
                      amax, scale, a.x, z.ldx, z.D, p.Dp, p.ldd, scaled ? ws + p.off_x : nullptr};
    if ((e = launch_ff_back(back, z.dtype, p.back_tile, s)) != hipSuccess) return e;

    FfProduct dx{}, dd{}, dg{};
    dx.a[0] = r.wg;
    dx.a[1] = r.wu;
    dx.lda[0] = r.ldg;
    dx.lda[1] = r.ldu;
    dx.b = dg.b = ws + p.off_grad;
    dx.b_step = dg.b_step = p.ldf * es;
    dx.ldb = dg.ldb = 2 * p.ldf * es;
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
    dx.scale = scale;
    dg.amax = amax;

    dg.a[0] = scaled ? ws + p.off_x : r.x;
    dg.lda[0] = scaled ? p.ldd * es : r.ldx;
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
    dd.lda[0] = p.ldf * es;
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

    if (p.all_tile >= 0) {
        if ((e = launch_ff_all(dx, dd, dg, z.dtype, p.all_tile, s)) != hipSuccess) return e;
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
