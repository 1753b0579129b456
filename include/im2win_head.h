/*
 * Training-head operators next to the im2win convolution, for AMD Instinct
 * MI355X (gfx950) -- C ABI, in the same library as im2win_conv2d.h.
 *
 * A convolution network's features (conv2d_fwd's y, in either of its layouts)
 * go through a layer norm over their channels, dropout, and a linear
 * classifier under softmax cross entropy; each operator has its gradient:
 *
 *   layer_norm_fwd / layer_norm_bwd     normalisation over the channels of each
 *                                       position, optionally followed by dropout
 *   dropout_fwd                         dropout from a counter-based generator
 *                                       (its own backward pass: apply it to dy)
 *   linear_xent_fwd / linear_xent_bwd   softmax cross entropy of the logits
 *                                       x w^T, which are never stored
 *
 * Pointers are DEVICE pointers the caller allocates and owns; `stream` is a
 * hipStream_t passed as void* (NULL: the default stream). The current device has
 * to be the one the pointers and the stream belong to. All work is enqueued on
 * `stream`; the calls return without synchronising, allocate nothing and
 * keep no state. Every argument is validated before anything is enqueued; on an
 * error nothing is launched and no output is touched (CONV2D_ERR_HIP: launches
 * of earlier steps of the same call may have been enqueued). Tensors need the
 * alignment of their element type (workspaces 256 bytes); rows that start on
 * 16-byte boundaries take the kernels' vector loads. Results are deterministic:
 * no atomics, so the same call gives the same bits. Calls that share a
 * workspace must be ordered by the caller. The calls may be captured into a
 * graph (kernel launches only, no memory operations).
 *
 * Statuses and element types are those of im2win_conv2d.h.
 */
#ifndef IM2WIN_HEAD_H
#define IM2WIN_HEAD_H

#include "im2win_conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- dropout --------------------------------------------------------------
 * Element i of the n elements belongs to counter block b = offset + i/8
 * (modulo 2^64). Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011) on counter (b low, b high, 0, 0) and
 * key (seed low, seed high) gives four 32-bit words; the 16-bit number u of the
 * block's element j = i%8 is word j/2's low half for even j, its high half for
 * odd j. With T = floor(p * 65536 + 0.5):
 *
 *   y[i] = u >= T ? x[i] * (65536 / (65536 - T)) : 0
 *
 * so the drop probability is p rounded to 1/65536 and the scale keeps the mean
 * exactly. A dropped element is 0 whatever x holds (infinities and NaN too);
 * T = 65536 drops everything. No mask is stored: the backward pass is the same
 * call on dy with the same p, seed and offset. */
typedef struct {
    int64_t n;                /* elements, >= 0                                  */
    int32_t dtype;            /* a conv2d_dtype_t: storage type of x and y       */
    int32_t reserved;         /* must be 0                                       */
    double p;                 /* drop probability in [0, 1]                      */
    uint64_t seed, offset;    /* key, and first counter block                    */
} dropout_desc_t;

/* y may be x itself. x * scale is formed in fp32 and rounded once. */
conv2d_status_t dropout_fwd(const dropout_desc_t *d, const void *x, void *y, void *stream);

/* ---- layer norm over channels ------------------------------------------------
 *   mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps)
 *   y = drop((x - mean) * rstd * weight[c] + bias[c])
 *
 * per position, with drop the dropout above over the elements in the order of
 * a contiguous y (the identity for dropout_p = 0), and
 *
 *   dz = drop(dy), g = dz * weight, xhat = (x - mean) * rstd
 *   dx = rstd * (g - sum_c g / C - xhat * sum_c (g * xhat) / C)
 *   dweight[c] = sum_positions dz * xhat,  dbias[c] = sum_positions dz
 *
 * NHWC: N positions of C contiguous channels (P = 1), row strides ldx, ldy,
 * lddx in elements (0: C). NCHW: N images of C planes of P positions,
 * contiguous (the strides must be 0). Statistics, sums and weight, bias and
 * their gradients are fp32; y and dx are rounded once. N may be 0 (dweight and
 * dbias are then 0). */
typedef struct {
    int64_t N, C, P;
    int64_t ldx;              /* NHWC row stride of x                            */
    int64_t ldy;              /* ... of y (forward) and dy (backward)            */
    int64_t lddx;             /* ... of dx                                       */
    int32_t dtype;            /* storage type of x and dx                        */
    int32_t y_dtype;          /* of y and dy: dtype, or any type if dtype is f32 */
    int32_t layout;           /* a conv2d_layout_t                               */
    int32_t reserved;         /* must be 0                                       */
    double eps;               /* >= 0                                            */
    double dropout_p;
    uint64_t seed, offset;
} layer_norm_desc_t;

/* weight, bias: fp32 [C], or NULL (1 and 0). mean, rstd: fp32, one per
 * position ([N] or [N][P]), or NULL both when no backward pass follows. */
conv2d_status_t layer_norm_fwd(const layer_norm_desc_t *d, const void *x, const float *weight,
                               const float *bias, void *y, float *mean, float *rstd, void *stream);

/* Bytes of workspace layer_norm_bwd needs (0 if d is invalid). */
size_t layer_norm_bwd_workspace_size(const layer_norm_desc_t *d);

/* mean, rstd as layer_norm_fwd wrote them. dweight, dbias: fp32 [C], or NULL
 * both for dx alone. */
conv2d_status_t layer_norm_bwd(const layer_norm_desc_t *d, const void *dy, const void *x,
                               const float *weight, const float *mean, const float *rstd, void *dx,
                               float *dweight, float *dbias, void *ws, void *stream);

/* ---- softmax cross entropy of a linear classifier -----------------------------
 *   l[i][v] = sum_d x[i][d] * w[v][d],  lse[i] = log sum_v exp(l[i][v])
 *   loss[i] = lse[i] - l[i][target[i]]
 *
 * and, for an upstream gradient grad[i] of loss[i],
 *
 *   G[i][v] = grad[i] * (exp(l[i][v] - lse[i]) - [v == target[i]])
 *   dx[i] = sum_v G[i][v] * w[v],  dw[v] = sum_i G[i][v] * x[i]
 *
 * A row whose target lies outside [0, V) is masked: loss, lse and dx are 0
 * there and it adds nothing to dw, whatever x holds in it. The logits are formed
 * tile by tile in fp32 and never stored; the backward pass forms them a
 * second time, in pieces of the classes, and holds one piece of G in the
 * workspace in the type of x (fp16: scaled by a power of two into the type's
 * range, which the largest finite grad of an unmasked row decides; half
 * precision: what that rounding takes from each row's target entry is added
 * back, and an offset that the class weights share still cancels in dx). dx and dw are accumulated in fp32 and rounded once. N may be
 * 0 (dw is then 0). */
typedef struct {
    int64_t N, V, D;          /* rows, classes, features                          */
    int64_t ldx, ldw;         /* row strides of x and w in elements (0: D)        */
    int32_t dtype;            /* storage type of x, w, dx and dw                  */
    int32_t reserved;         /* must be 0                                        */
} linear_xent_desc_t;

/* Limits: N <= 2^22, V <= 2^24, D, ldx, ldw <= 2^20. Where D and the row stride
 * are multiples of 16 bytes (8 half-precision or 4 fp32 elements) the rows are
 * read in place and x and w must start on a 16-byte boundary (backward: w
 * alone); other rows may start anywhere and are copied into the workspace first.
 *
 * Bytes of workspace linear_xent_fwd / linear_xent_bwd need (0 if d is
 * invalid, or when none is needed). */
size_t linear_xent_fwd_workspace_size(const linear_xent_desc_t *d);
size_t linear_xent_bwd_workspace_size(const linear_xent_desc_t *d);

/* target: int64 [N]. loss, lse: fp32 [N]. */
conv2d_status_t linear_xent_fwd(const linear_xent_desc_t *d, const void *x, const void *w,
                                const int64_t *target, float *loss, float *lse, void *ws, void *stream);

/* grad: fp32 [N]; lse as linear_xent_fwd wrote it. dx [N][D] and dw [V][D] are
 * contiguous and whole outputs. */
conv2d_status_t linear_xent_bwd(const linear_xent_desc_t *d, const float *grad, const void *x,
                                const void *w, const int64_t *target, const float *lse, void *dx, void *dw,
                                void *ws, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* IM2WIN_HEAD_H */
