// The tiled products' launches: tile shapes, what a launch of each takes, and the
// choice of tile and split.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

namespace im2win {

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }
inline int64_t elem(int dtype) { return dtype == 0 ? 4 : 2; }

// lets `kernel` take `bytes` of dynamic LDS on the current device, once per
// device (`done` has a bit for each)
inline hipError_t allow_lds(const void *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    const hipError_t e2 = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e2 == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e2;
}

// tile shapes of the products (contiguous index of the output x its rows)
enum ProductTile { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile32K = 3, kTile64x32 = 4, kTileNarrow = 5, kTiles = 6 };

// Time of one launch, from measurements of each tile shape (bf16 and fp32,
// 8192 x 16384 outputs over K 512 .. 4096, and single workgroups over K 8192):
// microseconds of a K stage with 1, 2, .. workgroups on a CU, and what a
// workgroup adds per tile. Half precision at K = 512, 1024, 4096 (TFLOP/s):
// 256 x 256 1079, 1168, 1418; 128 x 128 881, 984, 1163; 64 x 64 576, 669, 725;
// a lone 64 x 64 workgroup takes 0.30 us a stage, 128 x 128 0.69, 256 x 256 1.28.
struct TileShape {
    int64_t m, n;
    int per_cu;              // workgroups a CU holds
    double half[4], f32[4];  // us per stage with 1, 2, .. of them
    double fixed;            // us per tile before its epilogue
};
constexpr TileShape kShapes[5] = {{256, 256, 1, {1.42}, {7.3}, 4.3},
                                  {128, 128, 2, {0.69, 0.88}, {1.9, 3.7}, 2.7},
                                  {64, 64, 3, {0.30, 0.42, 0.53}, {0.48, 0.93, 1.4}, 1.3},
                                  {32, 32, 1, {0.28}, {0.60}, 2.5},              // K over four waves
                                  {64, 32, 4, {0.25, 0.30, 0.36, 0.42}, {0.30, 0.50, 0.73, 0.95}, 1.3}};
constexpr int64_t kCus = 256;

// microseconds of a product of M x N outputs over `stages` K stages that leaves
// out_bytes per output
inline double product_us(const TileShape &t, int64_t M, int64_t N, int64_t stages, int split, int dtype, int out_bytes,
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

// tile and split of a product whose K may be split (classes: of dw in the cross
// entropy, else 0)
inline void pick_product(int64_t M, int64_t N, int64_t stages, int dtype, int64_t classes, int *tile, int *split)
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

}  // namespace im2win
