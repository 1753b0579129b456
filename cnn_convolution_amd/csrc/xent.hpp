// The linear cross entropy's plan and the launchers of its kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "head_launch.hpp"

namespace im2win {

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

// tile shapes of the products (classes or features x rows or classes)
enum XentTile { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile32K = 3, kTile64x32 = 4, kTileNarrow = 5, kTiles = 6 };

// What a call does, from its sizes alone. Offsets are into the workspace.
struct XentPlan {
    int64_t Dp;              // D rounded up to whole 16-byte granules
    bool copy_x, copy_w;     // rows not made of 16-byte granules: padded copies
    int logits_tile;
    int64_t tiles_v;         // forward: partials per row
    int64_t piece;           // backward: classes per piece, row length of G
    int64_t rows_pad;        // rows of G
    int dx_tile, dx_split, dw_tile, dw_split;
    bool dx_direct;          // one piece and no split: dx straight from the product
    int64_t off_scale, off_t32, off_low, off_hits, off_rest, off_shared, off_some, off_x, off_w, off_partial, off_g,
        off_dx, off_dw, bytes;
};
XentPlan plan_xent_fwd(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype);
XentPlan plan_xent_bwd(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype);

// operands with 16-byte aligned rows, as the kernels read them
struct XentRows {
    const void *x, *w;
    int64_t ldx, ldw;        // bytes
};

struct LossArgs {
    XentRows r;
    int64_t N, V, Dp;
    const int64_t *target;
    float *loss;             // the target's logit
    float2 *partial;         // [tiles of classes][N]: (maximum, sum of exponentials around it)
};
hipError_t launch_xent_loss(const LossArgs &a, int dtype, int tile, hipStream_t s);

struct GradArgs {
    XentRows r;
    int64_t N, v0, P, Dp;    // classes v0 .. v0 + P - 1
    const int *t32;          // [rows_pad], -1: masked or past N
    const float *grad, *lse, *scale;   // scale[0]: S, or null (1)
    void *g;                 // [rows_pad][ldg]
    int64_t ldg;
    void *low;               // [N]: what rounding took from G at the target (half precision)
    uint8_t *hits;           // [piece / 32][rows_pad / 32]: whether a target lies in that block of G
    int64_t ldh;
    float *rest;             // [rest_blocks][ldr]: what rounding took from the other entries (half precision)
    int64_t ldr;
    const int *some;         // [somes]: whether the class weights share anything in 256 features; else no rest
    int somes;
};
// blocks of classes of `rest` that G of P classes leaves: one per wave and tile
int64_t rest_blocks(int tile, int64_t P);
hipError_t launch_xent_g(const GradArgs &a, int dtype, int tile, hipStream_t s);

struct ProductArgs {
    const void *a, *b;       // columns operand w or x; G
    int64_t lda, ldb;        // bytes
    int64_t M, n, k_a, k_b;  // output columns and rows; K values that exist in either
    int64_t K;
    int split;
    float *slab;             // [split][n][M] fp32, or null: straight into out
    bool add;                // slabs accumulate
    void *out;               // [n][M]
    const float *scale;      // scale[1]: 1/S, or null
    const int *t32;
    const void *low;
    const uint8_t *hits;     // dw
    int64_t ldh;
    int64_t v0;              // dw: first class of the piece
    const void *w;           // dx: for the rounding residual
    int64_t ldw;             // bytes
    const float *rest;       // dx in half precision: [blocks][ldr]
    int64_t ldr;
    int blocks;
    const float *shared;     // ... and [M rounded up to 256]: what the rows of w share
};
hipError_t launch_xent_dx(const ProductArgs &a, int dtype, int tile, hipStream_t s);
hipError_t launch_xent_dw(const ProductArgs &a, int dtype, int tile, hipStream_t s);
// both with 64 x 64 tiles
hipError_t launch_xent_both(const ProductArgs &dx, const ProductArgs &dw, int dtype, hipStream_t s);
// the slabs added, in order, into out; either may be null
hipError_t launch_xent_join(const ProductArgs *dx, const ProductArgs *dw, int dtype, hipStream_t s);

}  // namespace im2win
