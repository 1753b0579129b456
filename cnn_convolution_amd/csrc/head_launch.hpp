// Host-side launchers of the training-head kernels (layer norm, dropout,
// linear cross entropy). Arguments are validated by the callers in
// head_api.cpp; every launcher enqueues on `stream` and returns
// hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace im2win {

// Workgroups of `threads` that one launch may have: a grid of more than 2^32 threads is
// run modulo 2^32, without an error (one of 2^32 is refused). Kernels with more to do
// stride over the rest or are launched in parts.
constexpr int64_t max_groups(int threads) { return ((int64_t(1) << 32) - 1) / threads; }

// Dropout over elements numbered in 64 bits (see im2win_head.h): element i is
// kept when its 16-bit number is at least `threshold` (0: everything is kept)
// and multiplied by `scale`.
struct DropSpec {
    uint64_t seed, offset;
    uint32_t threshold;      // 0 .. 65536
    float scale;             // 65536 / (65536 - threshold), 0 where everything is dropped
};

hipError_t launch_dropout(const void *x, void *y, int64_t n, int dtype, const DropSpec &d, hipStream_t s);

struct NormArgs {
    const void *x, *dy;      // dy: backward only
    const float *weight, *bias;
    float *mean, *rstd;      // written forward (or null), read backward
    void *out;               // y forward, dx backward
    float *dweight, *dbias;  // backward, or null
    float *partial;          // backward workspace: [blocks][2][C]
    int64_t N, P;
    int C;
    int64_t ldx, ldy, ldo;   // NHWC row strides of x, of dy (backward) and of out
    int dtype, y_dtype;
    float eps;
    DropSpec drop;
};
hipError_t launch_norm_rows_fwd(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_rows_bwd(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_nchw_fwd(const NormArgs &a, hipStream_t s);
hipError_t launch_norm_nchw_bwd(const NormArgs &a, hipStream_t s);
// rows of the backward kernels' partial sums ([rows][2][C] floats)
int64_t norm_rows_partials(int64_t N, int64_t C);
int64_t norm_nchw_partials(int64_t N, int64_t C, int64_t P);

// ---- linear cross entropy ----
// Every product is formed as out[col][m] += sum_k A[m][k] B[col][k] with m the
// contiguous index of the output: the classes of a logit row, the features of
// a gradient row.
struct XentArgs {
    int64_t N, V, D, ldx, ldw;
    int dtype;
    const void *x, *w;
    const int64_t *target;
    const float *grad;       // backward: [N]
    float *loss, *lse;       // forward: written (loss holds the target's logit in between); backward: lse read
    void *dx, *dw;
    void *ws;
};
// workspace bytes (256-byte multiples) of the two passes
int64_t xent_fwd_ws_bytes(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype);
int64_t xent_bwd_ws_bytes(int64_t N, int64_t V, int64_t D, int64_t ldx, int64_t ldw, int dtype);
hipError_t launch_xent_fwd(const XentArgs &a, hipStream_t s);
hipError_t launch_xent_bwd(const XentArgs &a, hipStream_t s);

}  // namespace im2win
