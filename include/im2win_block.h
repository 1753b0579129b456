/*
 * Block operators of a training head, for AMD Instinct MI355X (gfx950) -- C ABI,
 * in the same library as im2win_conv2d.h and im2win_head.h.
 *
 * Between the features' first norm and the classifier a head may have blocks: a
 * gated feed-forward block on each position, joined to the residual stream by
 * a norm, a gate and a scale; its parameters are trained by AdamW:
 *
 *   feed_forward_fwd / feed_forward_bwd     act(x Wg^T) * (x Wu^T) through Wd^T
 *   residual_norm_fwd / residual_norm_bwd   the norm after a block, its gate, the
 *                                           residual sum, and the norm before the
 *                                           next block, in one pass
 *   adamw_step                              one step over many tensors, states in
 *                                           32 or in 8 bits
 *
 * Pointers, streams, workspaces, statuses and element types are as in
 * im2win_head.h: device pointers of the current device, everything enqueued on
 * `stream`, nothing allocated, kept or synchronised, every argument checked before
 * anything is enqueued, no sum whose order changes (the same call gives the same
 * bits), calls may be captured into a graph. Inputs and outputs must not overlap
 * unless said.
 */
#ifndef IM2WIN_BLOCK_H
#define IM2WIN_BLOCK_H

#include "im2win_conv2d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- gated feed-forward block ------------------------------------------------
 *   a = x Wg^T,  u = x Wu^T,  h = act(a) * u,  y = h Wd^T
 *
 * x [N][D], Wg and Wu [F][D], Wd [O][F], y [N][O], and for the gradient dy of y
 *
 *   dh = dy Wd,  da = dh * u * act'(a),  du = dh * act(a)
 *   dx = da Wg + du Wu,  dWg = da^T x,  dWu = du^T x,  dWd = dy^T h
 *
 * act: FF_SILU a / (1 + exp(-a)), FF_GELU a (1 + erf(a / sqrt 2)) / 2,
 * FF_GELU_TANH a (1 + tanh(sqrt(2/pi) (a + 0.044715 a^3))) / 2, FF_RELU max(a, 0)
 * (its slope at 0 is 0), FF_SIGMOID 1 / (1 + exp(-a)).
 *
 * All products are accumulated in fp32, a, u and dh are fp32 throughout; h, da and
 * du are rounded to the type of x where the matrix cores read them (fp16: an h beyond
 * that type's range is infinite; da and du are held times a power of two for each row, which
 * brings its largest finite |dy| into [1/16, 1/8), and x for the weights' gradients over
 * it). y of few rows is formed from an h of twice those digits: of at most 16 rows, and of
 * at most FF_ROWS where Wg's, Wu's or Wd's rows or row strides are no multiples of 16 bytes.
 * The outputs are rounded once. Limits: N <= 2^22; D, F, O and the row strides <= 2^20; sizes
 * whose tiles are more than one launch takes (weights' gradients of a terabyte and more)
 * are refused as an invalid descriptor. N = 0 gives zero weight gradients. */
enum { FF_SILU = 0, FF_GELU = 1, FF_GELU_TANH = 2, FF_RELU = 3, FF_SIGMOID = 4 };
enum { FF_ROWS = 64 };

typedef struct {
    int64_t N, D, F, O;
    int64_t ldx, ldg, ldu, ldd;   /* row strides of x, Wg, Wu, Wd in elements (0: D, D, D, F) */
    int64_t ldy;                  /* of y (forward) and dy (backward) (0: O)                  */
    int32_t dtype;                /* storage type of all tensors                              */
    int32_t act;
    int32_t reserved;             /* must be 0                                                */
    int32_t reserved2;            /* must be 0                                                */
} feed_forward_desc_t;

/* Rows and row strides that are multiples of 16 bytes are read in place and have
 * to start on a 16-byte boundary; other rows may start anywhere and are copied into the
 * workspace first, but for a forward pass of at most 16 rows, or of at most FF_ROWS in fp32
 * or where the weights' rows are such ones.
 *
 * saved: what feed_forward_bwd needs of the forward pass (act(a) and u act'(a) in fp32,
 * h), feed_forward_saved_size() bytes, 256-byte aligned; NULL when no backward pass
 * follows (feed_forward_fwd_workspace_size has to be asked with the same choice).
 * Sizes are 0 if d is invalid, or when nothing is needed. */
size_t feed_forward_saved_size(const feed_forward_desc_t *d);
size_t feed_forward_fwd_workspace_size(const feed_forward_desc_t *d, int32_t with_saved);
size_t feed_forward_bwd_workspace_size(const feed_forward_desc_t *d);

conv2d_status_t feed_forward_fwd(const feed_forward_desc_t *d, const void *x, const void *w_gate, const void *w_up,
                                 const void *w_down, void *y, void *saved, void *ws, void *stream);

/* dx [N][D], dw_gate, dw_up [F][D] and dw_down [O][F] are contiguous and whole
 * outputs. saved is only read; act(a) and the slopes are what it holds, so d->act is
 * checked and has no other effect. */
conv2d_status_t feed_forward_bwd(const feed_forward_desc_t *d, const void *dy, const void *x, const void *w_gate,
                                 const void *w_up, const void *w_down, const void *saved, void *dx, void *dw_gate,
                                 void *dw_up, void *dw_down, void *ws, void *stream);

/* ---- norms around a residual sum ----------------------------------------------
 * b is a block's output, r the residual stream it was taken from, [N] rows of C:
 *
 *   p   = norm(b) * post_weight + post_bias      (post = 0: p = b)
 *   out = residual_scale * r + branch_scale * gate[group] * p
 *   y   = norm(out) * weight + bias
 *
 * with norm(z) = (z - mean) * rstd, rstd = 1 / sqrt(sum (z - mean)^2 / C + eps)
 * (RN_LAYER) or mean = 0 (RN_RMS). gate: fp32 [groups][C], row i in group
 * i / (N / groups), or NULL (1). For the gradients dy of y and dout of out, with
 * xhat(z) = (z - mean) * rstd and through(g, z) = rstd * (g - [RN_LAYER: sum g / C] -
 * xhat(z) * sum (g * xhat(z)) / C):
 *
 *   t = dout + through(dy * weight, out),  dweight = sum dy * xhat(out),  dbias = sum dy
 *   dr = residual_scale * t,  dp = branch_scale * gate * t
 *   dgate[g] = sum_{rows of g} branch_scale * t * p
 *   db = through(dp * post_weight, b),  dpost_weight = sum dp * xhat(b),  dpost_bias = sum dp
 *   (post = 0: db = dp)
 *
 * y is formed from the unrounded out. Statistics, sums, gate, weights and biases
 * and their gradients are fp32 (a row whose squares add up to more than fp32 holds, values of
 * 10^17 and more, has rstd 0); out, y, dr and db are rounded once. */
enum { RN_LAYER = 0, RN_RMS = 1 };

typedef struct {
    int64_t N, C;
    int64_t groups;               /* of the gate: divides N; 0 where gate is NULL            */
    int64_t ldb, ldr, ldo, ldy;   /* row strides of b, r, out and y in elements (0: C)       */
    int64_t lddr, lddb, lddo, lddy; /* ... of dr, db, dout and dy (backward)                 */
    int32_t dtype;                /* storage type of r, out, dout and dr                     */
    int32_t branch_dtype;         /* of b, y, dy and db: dtype, or any type if dtype is f32  */
    int32_t kind, post;
    double eps, residual_scale, branch_scale;
} residual_norm_desc_t;

/* post_weight, post_bias, weight, bias: fp32 [C], or NULL (1 and 0). stats: fp32
 * [N][4], the mean and rstd of b, then of out (those of b are 0 without post), or
 * NULL when no backward pass follows. */
conv2d_status_t residual_norm_fwd(const residual_norm_desc_t *d, const void *b, const void *r, const float *gate,
                                  const float *post_weight, const float *post_bias, const float *weight,
                                  const float *bias, void *out, void *y, float *stats, void *stream);

size_t residual_norm_bwd_workspace_size(const residual_norm_desc_t *d);

/* out and stats as residual_norm_fwd wrote them. dout may be NULL (0). dgate
 * (only with a gate), dpost_weight, dpost_bias (only with post), dweight, dbias:
 * each may be NULL; the workspace is needed unless all are. */
conv2d_status_t residual_norm_bwd(const residual_norm_desc_t *d, const void *dy, const void *dout, const void *b,
                                  const void *out, const float *stats, const float *gate, const float *post_weight,
                                  const float *post_bias, const float *weight, void *dr, void *db, float *dgate,
                                  float *dpost_weight, float *dpost_bias, float *dweight, float *dbias, void *ws,
                                  void *stream);

/* ---- AdamW over many tensors ---------------------------------------------------
 * With g the gradient times grad_scale, per element, t the number of the step:
 *
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * in fp32 (8-bit states: m and v in fp64), p rounded once, and to `copy` where
 * there is one. 32-bit states: m, v fp32 [n].
 *
 * 8-bit states: blocks of 256 consecutive elements of a tensor share a scale each,
 * M = max |m| and V = max v of the new values, rounded to fp32; codes are int8 for
 * m and uint8 for v and stand for
 *
 *   m = sign(k) M (k / 127)^2,  v = V (k / 255)^4
 *
 * A value between two levels goes to the upper one (in magnitude) when 65536 times
 * its share of the interval exceeds a 16-bit number, so that its mean is the value:
 * rounded to the nearest, a state that moves by less than half a level a step would
 * not move at all. v > 0 goes to level 1 at least. Element i of a tensor has word
 * (first + i) % 4 of Philox4x32-10 on counter ((first + i) / 4, t) with key `seed`;
 * its low half decides m, its high half v. A block with an infinite or NaN m or v
 * gets the scale NaN. */
typedef struct {
    void *param;                  /* [n], updated                                   */
    const void *grad;             /* [n]                                            */
    void *copy;                   /* [n] of copy_dtype, or NULL                     */
    void *m, *v;                  /* [n]: fp32, or int8 and uint8                   */
    float *m_scale, *v_scale;     /* 8 bits: [ceil(n / 256)], else NULL             */
    int64_t n;
    int64_t first;                /* 8 bits: number of the first element, a multiple of 256 */
    int32_t param_dtype, grad_dtype, copy_dtype;
    int32_t reserved;             /* must be 0                                      */
    double lr, weight_decay;
} adamw_tensor_t;

typedef struct {
    int64_t count;                /* tensors, >= 0                                  */
    int32_t bits;                 /* of the states: 32 or 8                         */
    int32_t reserved;             /* must be 0                                      */
    double beta1, beta2, eps;     /* in [0, 1), [0, 1), >= 0                        */
    double grad_scale;
    uint64_t seed;                /* 8 bits                                         */
    int64_t step;                 /* t >= 1, or 0 where step_ptr is given           */
} adamw_desc_t;

/* tensors: host array of d->count entries, read before the call returns. The
 * parameters, copies, states and scales must not overlap (gradients may overlap
 * each other: they are read). Device
 * scalars for steps that are captured and replayed, or NULL: step_ptr (int64, t),
 * grad_scale_ptr (fp32, multiplies grad_scale), lr_ptr (fp32, multiplies every lr). */
conv2d_status_t adamw_step(const adamw_desc_t *d, const adamw_tensor_t *tensors, const int64_t *step_ptr,
                           const float *grad_scale_ptr, const float *lr_ptr, void *stream);

/* What n codes of 8-bit states stand for: blocks of 256 from the first on. */
conv2d_status_t adamw_values(int64_t n, const void *m, const void *v, const float *m_scale, const float *v_scale,
                             float *m_values, float *v_values, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* IM2WIN_BLOCK_H */
