// C ABI of the training-head operators (declared in include/im2win_head.h):
// argument checks, workspace sizes, and the choice of launcher.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "head_launch.hpp"
#include "im2win_head.h"

using namespace im2win;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;      // of one size
constexpr int64_t kMaxElems = int64_t(1) << 40;    // of one tensor: byte offsets stay within 64 bits

bool type_ok(int32_t t) { return t == CONV2D_F32 || t == CONV2D_F16 || t == CONV2D_BF16; }
int64_t esize(int32_t t) { return t == CONV2D_F32 ? 4 : 2; }
bool aligned(const void *p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % uintptr_t(a) == 0; }

conv2d_status_t hip_status(hipError_t e) { return e == hipSuccess ? CONV2D_OK : CONV2D_ERR_HIP; }

// p in [0, 1] (not NaN) -> the generator's threshold and scale
bool make_drop(double p, uint64_t seed, uint64_t offset, DropSpec *d)
{
    if (!(p >= 0.0 && p <= 1.0)) return false;
    d->threshold = uint32_t(std::floor(p * 65536.0 + 0.5));
    d->scale = d->threshold < 65536 ? float(65536.0 / double(65536 - d->threshold)) : 0.f;
    d->seed = seed;
    d->offset = offset;
    return true;
}

conv2d_status_t check_norm(const layer_norm_desc_t *d, NormArgs *a)
{
    if (!d) return CONV2D_ERR_NULL_POINTER;
    if (d->reserved != 0) return CONV2D_ERR_INVALID_DESC;
    if (!type_ok(d->dtype) || !type_ok(d->y_dtype)) return CONV2D_ERR_UNSUPPORTED;
    if (d->y_dtype != d->dtype && d->dtype != CONV2D_F32) return CONV2D_ERR_UNSUPPORTED;
    if (d->layout != CONV2D_NHWC && d->layout != CONV2D_NCHW) return CONV2D_ERR_UNSUPPORTED;
    if (d->N < 0 || d->C < 1 || d->P < 1) return CONV2D_ERR_INVALID_DESC;
    if (d->N >= kMaxDim || d->C >= kMaxDim / 16 || d->P >= kMaxDim) return CONV2D_ERR_INVALID_DESC;
    if (!(d->eps >= 0.0) || !std::isfinite(d->eps)) return CONV2D_ERR_INVALID_DESC;
    *a = NormArgs{};
    if (!make_drop(d->dropout_p, d->seed, d->offset, &a->drop)) return CONV2D_ERR_INVALID_DESC;
    a->ldx = d->ldx ? d->ldx : d->C;
    a->ldy = d->ldy ? d->ldy : d->C;
    a->ldo = d->lddx ? d->lddx : d->C;
    if (d->layout == CONV2D_NHWC) {
        if (d->P != 1 || a->ldx < d->C || a->ldy < d->C || a->ldo < d->C) return CONV2D_ERR_INVALID_DESC;
        for (int64_t ld : {a->ldx, a->ldy, a->ldo})
            if (ld > kMaxElems || (d->N && ld > kMaxElems / d->N)) return CONV2D_ERR_INVALID_DESC;
    } else {
        if (d->ldx || d->ldy || d->lddx) return CONV2D_ERR_INVALID_DESC;
        if (d->C > kMaxElems / d->P || (d->N && d->C * d->P > kMaxElems / d->N)) return CONV2D_ERR_INVALID_DESC;
    }
    a->N = d->N;
    a->C = int(d->C);
    a->P = d->P;
    a->dtype = d->dtype;
    a->y_dtype = d->y_dtype;
    a->eps = float(d->eps);
    return CONV2D_OK;
}

int64_t norm_partials(const layer_norm_desc_t &d)
{
    return d.layout == CONV2D_NHWC ? norm_rows_partials(d.N, d.C) : norm_nchw_partials(d.N, d.C, d.P);
}

conv2d_status_t check_xent(const linear_xent_desc_t *d, XentArgs *a)
{
    if (!d) return CONV2D_ERR_NULL_POINTER;
    if (d->reserved != 0) return CONV2D_ERR_INVALID_DESC;
    if (!type_ok(d->dtype)) return CONV2D_ERR_UNSUPPORTED;
    *a = XentArgs{};
    a->N = d->N;
    a->V = d->V;
    a->D = d->D;
    a->ldx = d->ldx ? d->ldx : d->D;
    a->ldw = d->ldw ? d->ldw : d->D;
    a->dtype = d->dtype;
    // tile offsets (256 rows of a stride) stay within 32 bits
    if (d->N < 0 || d->V < 1 || d->D < 1) return CONV2D_ERR_INVALID_DESC;
    if (d->N > (int64_t(1) << 22) || d->V > (int64_t(1) << 24) || d->D > (int64_t(1) << 20))
        return CONV2D_ERR_INVALID_DESC;
    if (a->ldx < d->D || a->ldw < d->D) return CONV2D_ERR_INVALID_DESC;
    if (a->ldx > (int64_t(1) << 20) || a->ldw > (int64_t(1) << 20)) return CONV2D_ERR_INVALID_DESC;
    return CONV2D_OK;
}

// rows of whole 16-byte granules are read as such; other rows are copied first
// and need only their element's alignment
bool rows_aligned(const void *p, int64_t D, int64_t ld, int32_t dtype)
{
    const int64_t es = esize(dtype), e = 16 / es;
    return aligned(p, D % e == 0 && ld % e == 0 ? 16 : es);
}

}  // namespace

extern "C" {

conv2d_status_t dropout_fwd(const dropout_desc_t *d, const void *x, void *y, void *stream)
{
    if (!d) return CONV2D_ERR_NULL_POINTER;
    DropSpec spec{};
    if (d->reserved != 0 || d->n < 0 || d->n > kMaxElems) return CONV2D_ERR_INVALID_DESC;
    if (!type_ok(d->dtype)) return CONV2D_ERR_UNSUPPORTED;
    if (!make_drop(d->p, d->seed, d->offset, &spec)) return CONV2D_ERR_INVALID_DESC;
    if (d->n == 0) return CONV2D_OK;
    if (!x || !y) return CONV2D_ERR_NULL_POINTER;
    if (!aligned(x, esize(d->dtype)) || !aligned(y, esize(d->dtype))) return CONV2D_ERR_MISALIGNED;
    return hip_status(launch_dropout(x, y, d->n, d->dtype, spec, static_cast<hipStream_t>(stream)));
}

conv2d_status_t layer_norm_fwd(const layer_norm_desc_t *d, const void *x, const float *weight, const float *bias,
                               void *y, float *mean, float *rstd, void *stream)
{
    NormArgs a;
    const conv2d_status_t st = check_norm(d, &a);
    if (st != CONV2D_OK) return st;
    if (d->N == 0) return CONV2D_OK;
    if (!x || !y || !mean != !rstd) return CONV2D_ERR_NULL_POINTER;
    if (!aligned(x, esize(d->dtype)) || !aligned(y, esize(d->y_dtype))) return CONV2D_ERR_MISALIGNED;
    for (const void *p : {static_cast<const void *>(weight), static_cast<const void *>(bias),
                          static_cast<const void *>(mean), static_cast<const void *>(rstd)})
        if (!aligned(p, 4)) return CONV2D_ERR_MISALIGNED;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.out = y;
    a.ldo = a.ldy;
    a.mean = mean;
    a.rstd = rstd;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(d->layout == CONV2D_NHWC ? launch_norm_rows_fwd(a, s) : launch_norm_nchw_fwd(a, s));
}

size_t layer_norm_bwd_workspace_size(const layer_norm_desc_t *d)
{
    NormArgs a;
    if (check_norm(d, &a) != CONV2D_OK) return 0;
    return size_t(norm_partials(*d) * 2 * d->C * 4);
}

conv2d_status_t layer_norm_bwd(const layer_norm_desc_t *d, const void *dy, const void *x, const float *weight,
                               const float *mean, const float *rstd, void *dx, float *dweight, float *dbias,
                               void *ws, void *stream)
{
    NormArgs a;
    const conv2d_status_t st = check_norm(d, &a);
    if (st != CONV2D_OK) return st;
    if (!dweight != !dbias) return CONV2D_ERR_NULL_POINTER;
    if (d->N == 0 && !dweight) return CONV2D_OK;
    if (d->N > 0 && (!dy || !x || !mean || !rstd || !dx)) return CONV2D_ERR_NULL_POINTER;
    if (dweight && !ws) return CONV2D_ERR_WORKSPACE;
    if (!aligned(x, esize(d->dtype)) || !aligned(dx, esize(d->dtype)) || !aligned(dy, esize(d->y_dtype)))
        return CONV2D_ERR_MISALIGNED;
    for (const float *p : {weight, mean, rstd, static_cast<const float *>(dweight), static_cast<const float *>(dbias)})
        if (!aligned(p, 4)) return CONV2D_ERR_MISALIGNED;
    if (!aligned(ws, 256)) return CONV2D_ERR_MISALIGNED;
    a.x = x;
    a.dy = dy;
    a.weight = weight;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.out = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.partial = dweight ? static_cast<float *>(ws) : nullptr;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(d->layout == CONV2D_NHWC ? launch_norm_rows_bwd(a, s) : launch_norm_nchw_bwd(a, s));
}

size_t linear_xent_fwd_workspace_size(const linear_xent_desc_t *d)
{
    XentArgs a;
    if (check_xent(d, &a) != CONV2D_OK) return 0;
    return size_t(xent_fwd_ws_bytes(a.N, a.V, a.D, a.ldx, a.ldw, a.dtype));
}

size_t linear_xent_bwd_workspace_size(const linear_xent_desc_t *d)
{
    XentArgs a;
    if (check_xent(d, &a) != CONV2D_OK) return 0;
    return size_t(xent_bwd_ws_bytes(a.N, a.V, a.D, a.ldx, a.ldw, a.dtype));
}

conv2d_status_t linear_xent_fwd(const linear_xent_desc_t *d, const void *x, const void *w, const int64_t *target,
                                float *loss, float *lse, void *ws, void *stream)
{
    XentArgs a;
    const conv2d_status_t st = check_xent(d, &a);
    if (st != CONV2D_OK) return st;
    if (d->N == 0) return CONV2D_OK;
    if (!x || !w || !target || !loss || !lse) return CONV2D_ERR_NULL_POINTER;
    if (!ws && linear_xent_fwd_workspace_size(d)) return CONV2D_ERR_WORKSPACE;
    if (!rows_aligned(x, a.D, a.ldx, a.dtype) || !rows_aligned(w, a.D, a.ldw, a.dtype) || !aligned(target, 8) ||
        !aligned(loss, 4) || !aligned(lse, 4) || !aligned(ws, 256))
        return CONV2D_ERR_MISALIGNED;
    a.x = x;
    a.w = w;
    a.target = target;
    a.loss = loss;
    a.lse = lse;
    a.ws = ws;
    return hip_status(launch_xent_fwd(a, static_cast<hipStream_t>(stream)));
}

conv2d_status_t linear_xent_bwd(const linear_xent_desc_t *d, const float *grad, const void *x, const void *w,
                                const int64_t *target, const float *lse, void *dx, void *dw, void *ws, void *stream)
{
    XentArgs a;
    const conv2d_status_t st = check_xent(d, &a);
    if (st != CONV2D_OK) return st;
    if (!w || !dw) return CONV2D_ERR_NULL_POINTER;
    if (d->N > 0 && (!grad || !x || !target || !lse || !dx)) return CONV2D_ERR_NULL_POINTER;
    if (!ws && linear_xent_bwd_workspace_size(d)) return CONV2D_ERR_WORKSPACE;
    const int64_t es = esize(d->dtype);
    if (!aligned(x, es) || !rows_aligned(w, a.D, a.ldw, a.dtype) || !aligned(dx, es) || !aligned(dw, es) || !aligned(grad, 4) ||
        !aligned(target, 8) || !aligned(lse, 4) || !aligned(ws, 256))
        return CONV2D_ERR_MISALIGNED;
    a.x = x;
    a.w = w;
    a.target = target;
    a.grad = grad;
    a.lse = const_cast<float *>(lse);
    a.dx = dx;
    a.dw = dw;
    a.ws = ws;
    return hip_status(launch_xent_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
