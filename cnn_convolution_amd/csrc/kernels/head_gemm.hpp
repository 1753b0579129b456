// Tiled matrix product of the linear cross entropy and the feed-forward block,
// out[n][m] = sum_k A[m][k] B[n][k], on the matrix cores with fp32 accumulation.
//
// A K stage is 128 bytes of K (64 half-precision or 32 fp32 values). Both tiles
// go from memory straight into LDS (global_load_lds_dwordx4, 1 KB per wave
// instruction, no registers, no LDS store), NST stages deep. An operand is
// stored in memory either with K contiguous ("rows": W and x for the logits, G
// for dx) or with its other index contiguous ("columns": w for dx, G and x for
// dw); its LDS image keeps that order:
//   rows     128 bytes per row; granule g (16 bytes) of row r in slot g ^ (r & 7)
//   columns  one K value's columns per LDS row; granule g of K row k in slot
//            g ^ swz(k), fetched transposed by ds_read_b64_tr_b16 (lane i of a
//            group of 16 receives column i of the four K rows the group's
//            addresses name), fp32 by plain 4-byte reads
// so that the fragment reads spread over all LDS banks. Either way a lane ends
// up with the same fragment: of row (column) lane%16, half precision the 8 K
// values 32h + 8(lane/16) .., fp32 the 4 values 16h + 4(lane/16) .., for half h
// of the stage.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../head_launch.hpp"
#include "lds_dma.hpp"

namespace im2win {

// BM x BN tile by WM x WN waves, NST stage buffers; per_cu: workgroups that a CU
// holds (LDS)
template <int BM_, int BN_, int WM_, int WN_, int NST_, int PER_CU>
struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_, per_cu = PER_CU;
    static constexpr int waves = WM * WN, threads = waves * 64, per_simd = waves * PER_CU / 4;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int a_bytes = BM * 128, b_bytes = BN * 128;
    static constexpr int lds_bytes = (a_bytes + b_bytes) * NST;
};
using C256 = TileCfg<256, 256, 2, 4, 2, 1>;
using C128 = TileCfg<128, 128, 2, 2, 2, 2>;
using C64 = TileCfg<64, 64, 2, 2, 3, 3>;
using C64x32 = TileCfg<64, 32, 2, 2, 3, 4>;
// for few rows, bound by the one read of W: four buffers in flight beat eight (1 row,
// 65536 x 2048 bf16 61.6 us, with eight 67.5; half as wide with two waves 65.3)
using CNarrow = TileCfg<128, 16, 4, 1, 4, 2>;

// Tiles of a launch at most: a tile's number plus a grid stays within an int. 2^22
// rows by 2^24 classes are that many tiles of 256 x 256.
constexpr int64_t kMaxTiles = int64_t(1) << 30;

// Workgroups of a launch over `tiles` tiles of `stages` K stages. Where a CU holds
// one workgroup, or the tiles are short, as many as the chip holds, each taking
// every grid-th tile and starting the next one's copies before its epilogue; else
// one per tile: a neighbour's products cover the epilogue, and the CUs that
// finish first take what is left. (A step with a workgroup per tile and so, 64798
// classes, 256 features, bf16: 69 rows, dw in two stages, 73.6 and 72.7 us; 200 rows, four
// stages, 109.1 and 106.0; 400 rows, logits in four, 158.5 and 154.1. More stages: no
// difference with 6, 8 or 16 as the limit.)
template <typename C>
inline int64_t grid_of(int64_t tiles, int64_t stages)
{
    const int64_t held = int64_t(C::per_cu) * 256;
    return (C::per_cu == 1 || stages <= 4) && tiles > held ? held : std::min(tiles, max_groups(C::threads));
}

// A whole 32 x 32 tile per wave, the four waves of a workgroup each with a quarter
// of K and stage buffers of its own (no barriers); for launches that could not
// fill the chip otherwise and whose K cannot be split over workgroups. Epi: how
// the waves hold the tile once their sums are joined.
struct C32K : TileCfg<32, 32, 1, 1, 4, 1> {
    using Wave = TileCfg<32, 32, 1, 1, 4, 1>;
    using Epi = TileCfg<32, 32, 2, 2, 4, 1>;
    static constexpr int groups = 4, threads = 256, per_simd = 1;
    static constexpr int lds_bytes = Wave::lds_bytes * groups;
};
template <typename C>
constexpr bool kSplitWaves = std::is_same<C, C32K>::value;
template <typename C>
struct EpiOf {
    using type = C;
};
template <>
struct EpiOf<C32K> {
    using type = C32K::Epi;
};

// where granules past the end of K are read from
__device__ __align__(16) static const uint4 zero_granule = {0, 0, 0, 0};

typedef __attribute__((address_space(3))) char *lds_ptr;
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint32x4_t __attribute__((ext_vector_type(4)));

// 16 bytes per lane from base + off (off per lane) to LDS byte address lds +
// 16*lane
__device__ __forceinline__ void copy_to_lds_at(const char *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}

struct GemmOperand {
    const void *p;
    int64_t ld;              // bytes between rows (rows) or K rows (columns), a multiple of 16
    int64_t count;           // rows or columns that exist; columns: a multiple of 16 bytes' worth
    int64_t k_end;           // K values that exist, zeros past them
};

// one operand's tile: TB rows or columns, of which `count` exist in memory from
// `base` on
template <typename T, int TB, int WAVES, bool COLS>
struct TileLoad {
    static constexpr int E = 16 / int(sizeof(T));                 // elements per granule
    static constexpr int KI = 128 / int(sizeof(T));               // K per stage
    static constexpr int blocks = TB / 8, per_wave = blocks < WAVES ? 1 : blocks / WAVES;
    static constexpr int GR = TB / E;                             // granules per K row (columns)
    static_assert(blocks <= WAVES ? WAVES % blocks == 0 : blocks % WAVES == 0, "blocks per wave");
    static_assert(!COLS || (GR >= 8 && GR <= 64), "columns per K row");

    const char *base;        // of this tile at K = 0
    int64_t step;            // bytes per stage
    uint32_t off[per_wave];  // per lane, of each block

    // columns: slot of granule g in K row k is g ^ swz(k). 16 columns are 2
    // (half precision) or 4 granules, kept together; the K rows that one read
    // touches (8q + 0..3 half precision, 4q fp32, q < 4) get different banks
    static __device__ __forceinline__ int swz(int k)
    {
        if constexpr (sizeof(T) == 4) return ((k >> 2) & 3) * 4 & (GR - 1);
        else if constexpr (GR == 8) return (((k >> 1) & 1) | ((k >> 3) & 1) << 1) * 2;
        else return ((k & 3) | ((k >> 3) & 1) << 2) * 2;
    }

    static __device__ __forceinline__ int block(int wave, int i) { return (wave + WAVES * i) % blocks; }

    __device__ __forceinline__ void init(const GemmOperand &op, int64_t first, int wave, int lane)
    {
        const char *p = static_cast<const char *>(op.p);
        const int64_t ld_bytes = op.ld, count = op.count;
        if constexpr (!COLS) first = first < count ? first : count - 1;   // a tile of padding alone
        const int n = int(count - first < TB ? count - first : TB);       // at least 1
        if constexpr (!COLS) {
            base = p + first * ld_bytes;
            step = 128;
#pragma unroll
            for (int i = 0; i < per_wave; ++i) {
                const int r = min(block(wave, i) * 8 + (lane >> 3), n - 1);
                off[i] = uint32_t(r) * uint32_t(ld_bytes) + (((lane & 7) ^ (lane >> 3)) << 4);
            }
        } else {
            base = p + first * int64_t(sizeof(T));
            step = KI * ld_bytes;
#pragma unroll
            for (int i = 0; i < per_wave; ++i) {
                const int k = krow(wave, lane, i);
                off[i] = uint32_t(k) * uint32_t(ld_bytes) + uint32_t(granule(lane, k, n)) * 16;
            }
        }
    }
    static __device__ __forceinline__ int krow(int wave, int lane, int i)
    {
        return block(wave, i) * (64 / GR) + lane / GR;
    }
    // source granule of this lane in K row k; columns past the last granule
    // read that one (n is a multiple of E: they are never stored)
    static __device__ __forceinline__ int granule(int lane, int k, int n)
    {
        return min((lane % GR) ^ swz(k), n / E - 1);
    }

    // copy i of this wave for whole stage s
    __device__ __forceinline__ void issue(int64_t s, int i, uint32_t lds, int wave) const
    {
        copy_to_lds_at(base + s * step, off[i], __builtin_amdgcn_readfirstlane(lds + block(wave, i) * 1024));
    }
    // the last stage of a K that ends inside it (left < KI values): zeros past it, for both
    // operands (beside the other's zeros a repeated infinite value would leave NaN)
    __device__ __forceinline__ void issue_tail(int64_t stage, int left, uint32_t lds, int wave, int lane) const
    {
        const char *b = base + stage * step;
#pragma unroll
        for (int i = 0; i < per_wave; ++i) {
            // left >= KI: the stage is whole
            const int k = COLS ? krow(wave, lane, i) : ((lane & 7) ^ (lane >> 3)) * E;
            const char *src = k < left ? b + off[i] : reinterpret_cast<const char *>(&zero_granule);
            copy_to_lds(src, __builtin_amdgcn_readfirstlane(lds + block(wave, i) * 1024));
        }
    }
};

// fragment addresses of one operand: byte offsets into its tile, of half 0
template <typename T, int TB, bool COLS>
struct FragRead {
    static constexpr int RB = TB * int(sizeof(T));                // columns: bytes per K row
    uint32_t o;
    int first;               // columns: this wave's first block of 16

    // first: this wave's first row or column of the tile, a multiple of 16
    __device__ __forceinline__ void init(int f, int lane)
    {
        first = f / 16;
        if constexpr (!COLS) {
            o = uint32_t(f + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
        } else if constexpr (sizeof(T) == 2) {
            const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);   // K row; the second read is 4 rows on
            o = uint32_t(k) * RB + ((lane & 3) >> 1) * 16 + (lane & 1) * 8;
            o += swizzle(k) << 4;
        } else {
            const int k = (lane >> 4) * 4;                        // K rows k .. k + 3
            o = uint32_t(k) * RB + (lane & 15) * 4;
            o += swizzle(k) << 4;
        }
    }
    static __device__ __forceinline__ uint32_t swizzle(int k) { return TileLoad<T, TB, 1, true>::swz(k); }

    // block i (16 rows or columns) of half h; tile: LDS address of the stage's tile
    __device__ __forceinline__ uint4 read(lds_ptr tile, int i, int h) const
    {
        if constexpr (!COLS) {
            // half 1 is granules 4 .. 7 before the swizzle: slot bit 2 flips
            typedef __attribute__((address_space(3))) const uint32x4_t *vp;
            return __builtin_bit_cast(uint4, *(vp)(tile + ((o ^ (h << 6)) + i * 2048)));
        } else if constexpr (sizeof(T) == 2) {
            const uint32_t a = (o ^ uint32_t((first + i) * 32)) + h * 32 * RB;
            typedef __attribute__((address_space(3))) short4_t *tp;
            const short4_t u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tp)(tile + a));
            const short4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tp)(tile + a + 4 * RB));
            const uint2 x = __builtin_bit_cast(uint2, u), y = __builtin_bit_cast(uint2, v);
            return uint4{x.x, x.y, y.x, y.y};
        } else {
            typedef __attribute__((address_space(3))) const uint32_t *wp;
            const uint32_t a = (o ^ uint32_t((first + i) * 64)) + h * 16 * RB;
            return uint4{*(wp)(tile + a), *(wp)(tile + a + RB), *(wp)(tile + a + 2 * RB), *(wp)(tile + a + 3 * RB)};
        }
    }
};

template <typename T>
__device__ __forceinline__ floatx4_t mfma_half(const uint4 &a, const uint4 &b, floatx4_t c)
{
    if constexpr (sizeof(T) == 4) {
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
        return c;
    } else {
        return mfma16x16x32<std::is_same<T, __bf16>::value>(a, b, c);
    }
}

// No further products (see tile_product).
struct NoExtra {
    template <typename R, typename A>
    __device__ __forceinline__ void run(int, R, A &)
    {
    }
};

// The product of one tile after another, acc[i][j]: 16 x 16 blocks of this wave's
// part of the tile; lane l holds m = 16i + 4(l/16) + v and n = 16j + l%16 of it.
// start() requests the first stages, run() multiplies; between a tile's run()
// and its epilogue the next tile is started, so its first stages arrive while
// the epilogue works on registers.
//
// A stage is 2 * FM steps, step t = (half t / FM, A block t % FM): FN products,
// and between them a share of everything else, so that neither wave of a SIMD
// issues a long run of reads or copies while the matrix core waits:
//   A fragments are read LA steps ahead into a ring, B fragments (one set per
//   half) two to a step ahead of their half;
//   at step BS every read of this stage is done: the barrier that waits for
//   them (and for the next stage's copies) frees its buffer, and the next
//   stage's fragments are read from there on;
//   the copies of stage s + NST into that buffer go out one share per step from
//   BS on, into the next stage's first steps (64 KB take the CU's vector
//   memory path 1024 cycles of a stage's 2048).
// 256 x 256 tiles, bf16: 1.36 us per 64-wide stage, 1540 TFLOP/s (without the
// copies 1700, without the LDS reads 1580: what is left is issue and power).
// LoadA: what brings A's tile into LDS, one operand's unless said.
template <typename T, typename C, bool ACOLS, bool BCOLS, typename LoadA = TileLoad<T, C::BM, C::waves, ACOLS>>
struct TilePipe {
    static constexpr int KI = 128 / int(sizeof(T)), FM = C::FM, FN = C::FN, NST = C::NST;
    static constexpr int STEPS = 2 * FM;
    static constexpr int LA = FM >= 8 ? 4 : FM >= 4 ? 3 : 2;
    static constexpr int BS = STEPS - LA + 1;
    static constexpr int R = FM >= 8 ? 8 : 4;                 // ring of A fragments
    static constexpr int B1 = FM / 2 - 1;                     // first step that reads half 1's B
    static_assert(STEPS % R == 0 && LA + 1 <= R, "ring");

    const int lane, wave;
    const lds_ptr sm;        // the A buffers first, then the B buffers
    const uint32_t sbase;
    LoadA la;
    TileLoad<T, C::BN, C::waves, BCOLS> lb;
    FragRead<T, C::BM, ACOLS> ra;
    FragRead<T, C::BN, BCOLS> rb;
    int64_t a_end, b_end;    // K values of either operand
    int s0, s1;              // K stages [s0, s1)

    static constexpr int UA = decltype(la)::per_wave, D = UA + decltype(lb)::per_wave;   // copies per wave and stage
    static constexpr int PER = (D + FM - 1) / FM;             // copies per step
    static constexpr int TAIL = (STEPS - BS) * PER < D ? (STEPS - BS) * PER : D;   // copies that go out from BS on

    static constexpr bool SOLO = kSplitWaves<C>;              // a wave by itself
    // Tiles of few rows, whose few logits a library sums in many parts, add up RUN
    // stages at a time: in one chain the logit of a row's target, a sum of mostly
    // positive terms, loses half a bit per doubling of K (3 rows, 13948 classes, 1408
    // features, fp32: loss 1.6e-6 off in one chain, 1.7e-7 so). Time: 1 row, 20000
    // classes, 1024 features, fp32 19.3 and 20.4 us, nothing elsewhere; with 64 x 64
    // tiles too 3000 rows, 300 classes took 152 and 161.
    static constexpr bool PARTS = FM * FN <= 2;
    static constexpr int RUN = 4;

    __device__ __forceinline__ TilePipe(char *smem)
        : lane(threadIdx.x & 63), wave(SOLO ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
          sm((lds_ptr)(SOLO ? smem + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (C::a_bytes + C::b_bytes) * NST
                            : smem)),
          sbase(__builtin_amdgcn_readfirstlane(uint32_t(reinterpret_cast<uintptr_t>(sm))))
    {
        ra.init(wave % C::WM * (C::BM / C::WM), lane);
        rb.init(wave / C::WM * (C::BN / C::WN), lane);
    }

    static __device__ __forceinline__ void sync()
    {
        if constexpr (SOLO) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0) only
            asm volatile("" ::: "memory");
        } else {
            stage_barrier();
        }
    }

    __device__ __forceinline__ void request(int s, int buf)
    {
        const uint32_t a = sbase + buf * C::a_bytes, b = sbase + NST * C::a_bytes + buf * C::b_bytes;
        la.issue_tail(s, int(min(a_end - int64_t(s) * KI, int64_t(KI))), a, wave, lane);
        lb.issue_tail(s, int(min(b_end - int64_t(s) * KI, int64_t(KI))), b, wave, lane);
    }
    __device__ __forceinline__ void copy(int u, int s, int buf)      // copy u of whole stage s
    {
        if (u < UA)
            la.issue(s, u, sbase + buf * C::a_bytes, wave);
        else
            lb.issue(s, u - UA, sbase + NST * C::a_bytes + buf * C::b_bytes, wave);
    }

    // The buffers are free (run() has ended or not begun).
    template <typename OpA>
    __device__ __forceinline__ void start(const OpA &A, const GemmOperand &B, int64_t m0, int64_t n0, int first,
                                          int end)
    {
        s0 = first;
        s1 = end;
        a_end = A.k_end;
        b_end = B.k_end;
        la.init(A, m0, wave, lane);
        lb.init(B, n0, wave, lane);
#pragma unroll
        for (int s = 0; s < NST; ++s)
            if (s0 + s < s1) request(s0 + s, s);
    }

    // since: vector memory operations that each wave is known to have issued
    // since start() (no more than it has). extra.run(s, read, acc) may add products
    // of stage s's A fragments, read(i, h) for block i of half h. clear: acc starts at 0,
    // else the products are added to it.
    template <int SINCE, typename Extra>
    __device__ __forceinline__ void run(bool since, floatx4_t (&acc)[C::FM][C::FN], Extra &extra, bool clear = true)
    {
        const int whole = int(min(a_end, b_end) / KI);        // stages that both operands fill
        const int last = s1 - 1;
        if (clear) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        }

        floatx4_t total[PARTS ? FM : 1][PARTS ? FN : 1] = {};
        auto add_up = [&](bool clear) {
            if constexpr (PARTS)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        total[i][j] += acc[i][j];
                        acc[i][j] = clear ? floatx4_t{0.f, 0.f, 0.f, 0.f} : total[i][j];
                    }
        };

        uint4 ar[R], br[2][FN];
        auto read_a = [&](int u, int buf) { ar[u % R] = ra.read(sm + buf * C::a_bytes, u % FM, u % STEPS / FM); };
        auto read_b = [&](int j, int h, int buf) { br[h][j] = rb.read(sm + NST * C::a_bytes + buf * C::b_bytes, j, h); };

        static_assert(D * (NST - 1) + SINCE < 64, "wait count");
        if (last - s0 < NST - 1)
            wait_vm<0>();
        else if (SINCE > 0 && since)
            wait_vm<D * (NST - 1) + SINCE>();
        else
            wait_vm<D * (NST - 1)>();
        sync();
#pragma unroll
        for (int j = 0; j < FN; ++j) read_b(j, 0, 0);
#pragma unroll
        for (int u = 0; u < LA; ++u) read_a(u, 0);
        int buf = 0, prev = 0;
        bool pending = false;                                 // copies TAIL .. of stage s - 1 + NST are left
        for (int s = s0; s < s1; ++s) {
            const int next = buf + 1 == NST ? 0 : buf + 1;
            bool now = false;
            extra.run(s, [&](int i, int h) { return ra.read(sm + buf * C::a_bytes, i, h); }, acc);
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                if (t == BS) {
                    if (NST > 2 && s + NST - 1 <= last)
                        wait_vm<D * (NST - 2)>();
                    else
                        wait_vm<0>();
                    sync();
                    now = s + NST <= last;
                    if (now && s + NST >= whole) {
                        request(s + NST, buf);
                        now = false;
                    }
                }
                if (t >= BS) {
                    if (now) {
#pragma unroll
                        for (int u = (t - BS) * PER; u < (t - BS + 1) * PER && u < TAIL; ++u) copy(u, s + NST, buf);
                    }
                } else if (TAIL + t * PER < D) {
                    if (pending) {
#pragma unroll
                        for (int u = TAIL + t * PER; u < TAIL + (t + 1) * PER && u < D; ++u)
                            copy(u, s - 1 + NST, prev);
                    }
                }
                // after the last stage the reads from `next` find no stage there: unused
                if (t + LA < STEPS) read_a(t + LA, buf);
                if (t == BS) {
                    read_a(STEPS, next);
                    read_a(STEPS + 1, next);
                }
                if (t > BS) read_a(t + LA, next);
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    if (t >= B1 && t < FM && j / 2 == t - B1) read_b(j, 1, buf);
                    if (t >= BS && j / 2 == t - BS) read_b(j, 0, next);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[t % FM][j] = mfma_half<T>(ar[t % R], br[t / FM][j], acc[t % FM][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
            pending = now;
            prev = buf;
            buf = next;
            if (PARTS && (s - s0) % RUN == RUN - 1) add_up(true);
        }
        add_up(false);
        wait_vm<0>();
        sync();                   // no wave reads the buffers any more
    }
};

// The four waves' sums of C32K's tile added in order: on return wave w holds block
// (w % 2, w / 2) as its one block. smem: the stage buffers, no longer in use.
template <typename C>
__device__ __forceinline__ void join_waves(char *smem, const floatx4_t (&acc)[C::FM][C::FN], floatx4_t (&out)[1][1])
{
    floatx4_t *part = reinterpret_cast<floatx4_t *>(smem);    // [wave][block][lane], a wave's own buffers first
    constexpr int STRIDE = C::Wave::lds_bytes / int(sizeof(floatx4_t));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) part[wave * STRIDE + (j * 2 + i) * 64 + lane] = acc[i][j];
    __syncthreads();
    floatx4_t t = part[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) t += part[w * STRIDE + wave * 64 + lane];
    out[0][0] = t;
    __syncthreads();                           // the buffers may be written again
}

// 8 consecutive values of m per lane instead of 4: blocks i and i + 1 of a column
// exchanged between neighbouring rows of 16 lanes, so that a half-precision store
// is 16 bytes. Afterwards lane row q holds m = 16(i + q%2) + 8(q/2) .. + 7.
template <typename T>
__device__ __forceinline__ uint4 pair_blocks(const floatx4_t &a, const floatx4_t &b)
{
    typedef T pair __attribute__((ext_vector_type(2)));
    const auto pack = [](float u, float v) {
        return __builtin_bit_cast(uint32_t, pair{static_cast<T>(u), static_cast<T>(v)});
    };
    const auto x = __builtin_amdgcn_permlane16_swap(pack(a[0], a[1]), pack(b[0], b[1]), false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(pack(a[2], a[3]), pack(b[2], b[3]), false, false);
    return uint4{x[0], y[0], x[1], y[1]};
}

// workgroup -> (m, n) tile: each XCD gets a contiguous range of tiles, walked
// in strips of 8 n tiles, so the tiles it runs at a time share their panels in
// its L2
__device__ __forceinline__ void strip_tile(int b, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int G = tiles_m * tiles_n, per = G >> 3, rem = G & 7, x = b & 7;
    const int t = x * per + min(x, rem) + (b >> 3);
    const int strip = t / (tiles_m * 8), r = t - strip * tiles_m * 8;
    const int w = min(8, tiles_n - strip * 8);
    tm = r / w;
    tn = strip * 8 + r - tm * w;
}

}  // namespace im2win
