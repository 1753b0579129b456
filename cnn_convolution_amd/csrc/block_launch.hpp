// Host-side launchers of the block kernels (feed-forward block, norms around a
// residual sum, AdamW). Arguments are validated by the callers in block_api.cpp;
// every launcher enqueues on `stream` and returns hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace im2win {

// ---- feed-forward block ----
struct FfSizes {
    int64_t N, D, F, O, ldx, ldg, ldu, ldd, ldy;   // strides in elements
    int dtype, act;
};
struct FfArgs {
    FfSizes z;
    const void *x, *wg, *wu, *wd;
    void *y;                 // forward
    void *saved;             // forward: or null
    void *ws;
    const void *dy;          // backward
    void *dx, *dwg, *dwu, *dwd;
};
int64_t ff_saved_bytes(const FfSizes &z);
// of workspace; -1: a launch would have more tiles than one can
int64_t ff_fwd_ws_bytes(const FfSizes &z, bool saved);
int64_t ff_bwd_ws_bytes(const FfSizes &z);
hipError_t launch_ff_fwd(const FfArgs &a, hipStream_t s);
hipError_t launch_ff_bwd(const FfArgs &a, hipStream_t s);

// ---- norms around a residual sum ----
struct ResNormArgs {
    const void *b, *r;       // r: forward
    void *out;               // written forward, read backward
    void *y;                 // forward
    float *stats;            // [N][4], written forward (or null), read backward
    const float *gate, *pw, *pb, *w, *bias;
    const void *dy, *dout;   // backward; dout may be null
    void *dr, *db;
    float *dgate, *dpw, *dpb, *dw, *dbias;
    void *ws;
    int64_t N, rows;         // rows: of a gate's group
    int64_t groups;
    int C;
    int64_t ldb, ldr, ldo, ldy, lddr, lddb, lddo, lddy;
    int dtype, branch_dtype;
    int layer, post;         // 0 or 1
    float eps, rs, bs;
};
int64_t res_norm_bwd_ws_bytes(int64_t N, int64_t C, int64_t groups);
hipError_t launch_res_norm_fwd(const ResNormArgs &a, hipStream_t s);
hipError_t launch_res_norm_bwd(const ResNormArgs &a, hipStream_t s);

// ---- AdamW ----
struct AdamTensor {
    void *p;
    const void *g;
    void *copy, *m, *v;
    float *ms, *vs;
    int64_t n, first;
    float lr, decay;
    int32_t end;             // chunks of this launch up to and with this tensor's
    int8_t pt, gt, ct, pad;
};
constexpr int kAdamTensors = 40;               // of a launch: its arguments stay below 4 KB
struct AdamArgs {
    const int64_t *step_ptr;
    const float *grad_scale_ptr, *lr_ptr;
    double beta1, beta2;
    double rate;             // 1 / (1 - beta1^step), unless step_ptr gives the step
    int64_t step;
    uint64_t seed;
    float root;              // 1 / sqrt(1 - beta2^step), likewise
    float eps, grad_scale;
    int count;
    AdamTensor t[kAdamTensors];
};
constexpr int64_t adam_chunk(int bits) { return bits == 8 ? 1024 : 2048; }   // elements of a workgroup
hipError_t launch_adamw(const AdamArgs &a, int bits, hipStream_t s);
hipError_t launch_adamw_values(int64_t n, const void *m, const void *v, const float *ms, const float *vs, float *mo,
                               float *vo, hipStream_t s);

}  // namespace im2win
