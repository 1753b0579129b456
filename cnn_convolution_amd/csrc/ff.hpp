// The feed-forward block's plan and the launchers of its tiled products.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "block_launch.hpp"
#include "tile_launch.hpp"

namespace im2win {

// act(a) and u act'(a), the factors of dh in du and da, as the matrix cores leave them:
// fp32 blocks of 16 x 16, [row / 16][f / 16][two][lane][4] for whole tiles of 256 rows
// and features, lane l holding f = 4(l/16) + v and row l%16. Written (where rows and
// features exist) and read by the same lanes, 1 KB at a time.
struct FfSaved {
    float *pre;
    int64_t fblocks;
    void *h;                 // [rows_pad] rows of Fp, zeros past N and F
    int64_t ldh;             // elements between them: whole cache lines
};

// h (and with `pre` the factors) of rows 0 .. rows_pad - 1
struct FfGate {
    const void *x, *wg, *wu;
    int64_t ldx, ldg, ldu;   // bytes
    int64_t N, F, Dp, rows_pad, Fp;
    FfSaved to;              // pre: or null
    int act;
};
hipError_t launch_ff_gate(const FfGate &a, int dtype, int tile, hipStream_t s);

// da and du, each [rows_pad] rows of Fp with zeros past N and F, side by side in rows of
// 2 from.ldh; fp16: times their row's scale, and x the other way for the weights' gradients
struct FfBack {
    const void *dy, *wd;
    int64_t lddy, ldd;       // bytes
    int64_t N, F, O, Op, rows_pad, Fp;
    FfSaved from;
    void *g;
    // fp16 (see ff_common.hpp):
    const float *amax;       // [2][kAmaxParts]: of |dy|, of |x|
    const float *scale;      // [N]: of the rows of da and du
    const void *x;           // its rows as the caller has them
    int64_t ldx, D, Dp, ldt; // elements
    void *to_x;              // [N] rows of Dp, ldt apart: x times what its row's scale leaves
};
hipError_t launch_ff_back(const FfBack &a, int dtype, int tile, hipStream_t s);
constexpr int kAmaxParts = 256;

// out[n][m] = sum over segments and k of a[seg] times b: the products that leave an
// output. a: rows ([m][k], y) or columns ([k][m]); b: rows ([n][k], y and dx) or
// columns ([k][n], the weight gradients).
struct FfProduct {
    const void *a[2];        // per segment of K
    int64_t lda[2], ldb;     // bytes
    const void *b;
    int64_t b_step;          // bytes from b's part of a segment or output to the next one's
    int64_t M, a_count;      // outputs, and what exists of a
    int64_t n, b_count;      // rows of an output, and what exists of b
    int64_t K, k_a, k_b;     // of a segment
    int segs, outs;          // 1 or 2; outs 2: two outputs of n rows each
    int split;
    float *slab;             // [split][outs n][M] fp32, or null
    void *out[2];
    int64_t ldo;             // elements
    const float *amax;       // the outputs are divided by the scales it gives, or null
    const float *scale;      // or each row by its own (one output), or null
};
hipError_t launch_ff_y(const FfProduct &p, int dtype, int tile, hipStream_t s);
hipError_t launch_ff_dx(const FfProduct &p, int dtype, int tile, hipStream_t s);
hipError_t launch_ff_dw(const FfProduct &p, int dtype, int tile, hipStream_t s);
// dx, dw_down and dw_gate with dw_up in one launch, tiles of 128 or 64
hipError_t launch_ff_all(const FfProduct &dx, const FfProduct &dwd, const FfProduct &dwgu, int dtype, int tile,
                         hipStream_t s);
// the slabs of up to three products added in order
hipError_t launch_ff_join(const FfProduct *p, int count, int dtype, hipStream_t s);

// few rows: h in two parts (half precision), h itself and `lo` [N][ldh]; with a `pre` the
// factors, and h with its zero rows
struct FfRows {
    const void *x, *wg, *wu, *wd;
    int64_t ldx, ldg, ldu, ldd, ldy;   // elements
    int64_t N, D, F, O, Fp;
    FfSaved to;
    void *lo, *y;
    int act;
    int blocks;              // of 16 rows to write
    float *slab;             // y's sums over parts of K, where it is split
    int *count;              // [counts] of parts that are there, cleared by the gate's launch
    int counts;
};

}  // namespace im2win
