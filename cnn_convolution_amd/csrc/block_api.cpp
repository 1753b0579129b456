// C ABI of the block operators (declared in include/im2win_block.h): argument
// checks, workspace sizes, and the choice of launcher.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "block_launch.hpp"
#include "head_launch.hpp"
#include "im2win_block.h"

using namespace im2win;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;    // of one tensor: byte offsets stay within 64 bits

bool type_ok(int32_t t) { return t == CONV2D_F32 || t == CONV2D_F16 || t == CONV2D_BF16; }
int64_t esize(int32_t t) { return t == CONV2D_F32 ? 4 : 2; }
// (a number that fp32 does not hold is an infinity in the kernels)
bool finite32(double v) { return std::isfinite(float(v)); }
bool aligned(const void *p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % uintptr_t(a) == 0; }

conv2d_status_t hip_status(hipError_t e) { return e == hipSuccess ? CONV2D_OK : CONV2D_ERR_HIP; }

// ---- feed-forward block ----

conv2d_status_t check_ff(const feed_forward_desc_t *d, FfSizes *z)
{
    if (!d) return CONV2D_ERR_NULL_POINTER;
    if (d->reserved != 0 || d->reserved2 != 0) return CONV2D_ERR_INVALID_DESC;
    if (!type_ok(d->dtype) || d->act < FF_SILU || d->act > FF_SIGMOID) return CONV2D_ERR_UNSUPPORTED;
    constexpr int64_t kMax = int64_t(1) << 20;     // tile offsets (256 rows of a stride) stay within 32 bits
    if (d->N < 0 || d->N > int64_t(1) << 22) return CONV2D_ERR_INVALID_DESC;
    for (int64_t v : {d->D, d->F, d->O})
        if (v < 1 || v > kMax) return CONV2D_ERR_INVALID_DESC;
    *z = FfSizes{d->N, d->D, d->F, d->O, d->ldx ? d->ldx : d->D, d->ldg ? d->ldg : d->D, d->ldu ? d->ldu : d->D,
                 d->ldd ? d->ldd : d->F, d->ldy ? d->ldy : d->O, d->dtype, d->act};
    if (z->ldx < d->D || z->ldg < d->D || z->ldu < d->D || z->ldd < d->F || z->ldy < d->O)
        return CONV2D_ERR_INVALID_DESC;
    for (int64_t v : {z->ldx, z->ldg, z->ldu, z->ldd, z->ldy})
        if (v > kMax) return CONV2D_ERR_INVALID_DESC;
    return CONV2D_OK;
}

// rows of whole 16-byte granules are read as such; other rows are copied first and
// need only their element's alignment
bool rows_aligned(const void *p, int64_t D, int64_t ld, int32_t dtype)
{
    const int64_t es = esize(dtype), e = 16 / es;
    return aligned(p, D % e == 0 && ld % e == 0 ? 16 : es);
}

bool ff_inputs_aligned(const FfSizes &z, const void *x, const void *wg, const void *wu, const void *wd)
{
    return rows_aligned(x, z.D, z.ldx, z.dtype) && rows_aligned(wg, z.D, z.ldg, z.dtype) &&
           rows_aligned(wu, z.D, z.ldu, z.dtype) && rows_aligned(wd, z.F, z.ldd, z.dtype);
}

// ---- norms around a residual sum ----

conv2d_status_t check_res_norm(const residual_norm_desc_t *d, ResNormArgs *a)
{
    if (!d) return CONV2D_ERR_NULL_POINTER;
    if (!type_ok(d->dtype) || !type_ok(d->branch_dtype)) return CONV2D_ERR_UNSUPPORTED;
    if (d->branch_dtype != d->dtype && d->dtype != CONV2D_F32) return CONV2D_ERR_UNSUPPORTED;
    if (d->kind != RN_LAYER && d->kind != RN_RMS) return CONV2D_ERR_UNSUPPORTED;
    if (d->post != 0 && d->post != 1) return CONV2D_ERR_INVALID_DESC;
    if (d->N < 0 || d->N >= int64_t(1) << 31 || d->C < 1 || d->C >= int64_t(1) << 27) return CONV2D_ERR_INVALID_DESC;
    if (d->groups < 0 || (d->groups > 0 && (d->N % d->groups != 0 || d->C > kMaxElems / d->groups)))
        return CONV2D_ERR_INVALID_DESC;
    if (d->N > 0 && d->groups > d->N) return CONV2D_ERR_INVALID_DESC;
    for (double v : {d->residual_scale, d->branch_scale})
        if (!finite32(v)) return CONV2D_ERR_INVALID_DESC;
    if (!(d->eps >= 0.0) || !finite32(d->eps)) return CONV2D_ERR_INVALID_DESC;
    *a = ResNormArgs{};
    const auto stride = [&](int64_t ld) { return ld ? ld : d->C; };
    a->ldb = stride(d->ldb);
    a->ldr = stride(d->ldr);
    a->ldo = stride(d->ldo);
    a->ldy = stride(d->ldy);
    a->lddr = stride(d->lddr);
    a->lddb = stride(d->lddb);
    a->lddo = stride(d->lddo);
    a->lddy = stride(d->lddy);
    for (int64_t ld : {a->ldb, a->ldr, a->ldo, a->ldy, a->lddr, a->lddb, a->lddo, a->lddy})
        if (ld < d->C || ld > kMaxElems || (d->N && ld > kMaxElems / d->N)) return CONV2D_ERR_INVALID_DESC;
    a->N = d->N;
    a->C = int(d->C);
    a->groups = d->groups;
    a->rows = d->groups ? d->N / d->groups : d->N;
    a->dtype = d->dtype;
    a->branch_dtype = d->branch_dtype;
    a->layer = d->kind == RN_LAYER;
    a->post = d->post;
    a->eps = float(d->eps);
    a->rs = float(d->residual_scale);
    a->bs = float(d->branch_scale);
    return CONV2D_OK;
}

}  // namespace

extern "C" {

size_t feed_forward_saved_size(const feed_forward_desc_t *d)
{
    FfSizes z;
    return check_ff(d, &z) == CONV2D_OK ? size_t(ff_saved_bytes(z)) : 0;
}

size_t feed_forward_fwd_workspace_size(const feed_forward_desc_t *d, int32_t with_saved)
{
    FfSizes z;
    return check_ff(d, &z) == CONV2D_OK ? size_t(std::max<int64_t>(ff_fwd_ws_bytes(z, with_saved != 0), 0)) : 0;
}

size_t feed_forward_bwd_workspace_size(const feed_forward_desc_t *d)
{
    FfSizes z;
    return check_ff(d, &z) == CONV2D_OK ? size_t(std::max<int64_t>(ff_bwd_ws_bytes(z), 0)) : 0;
}

conv2d_status_t feed_forward_fwd(const feed_forward_desc_t *d, const void *x, const void *w_gate, const void *w_up,
                                 const void *w_down, void *y, void *saved, void *ws, void *stream)
{
    FfArgs a{};
    const conv2d_status_t st = check_ff(d, &a.z);
    if (st != CONV2D_OK) return st;
    if (d->N == 0) return CONV2D_OK;
    if (!x || !w_gate || !w_up || !w_down || !y) return CONV2D_ERR_NULL_POINTER;
    const int64_t need = ff_fwd_ws_bytes(a.z, saved != nullptr);
    if (need < 0) return CONV2D_ERR_INVALID_DESC;
    if (!ws && need) return CONV2D_ERR_WORKSPACE;
    if (!ff_inputs_aligned(a.z, x, w_gate, w_up, w_down) || !aligned(y, esize(d->dtype)) || !aligned(saved, 256) ||
        !aligned(ws, 256))
        return CONV2D_ERR_MISALIGNED;
    a.x = x;
    a.wg = w_gate;
    a.wu = w_up;
    a.wd = w_down;
    a.y = y;
    a.saved = saved;
    a.ws = ws;
    return hip_status(launch_ff_fwd(a, static_cast<hipStream_t>(stream)));
}

conv2d_status_t feed_forward_bwd(const feed_forward_desc_t *d, const void *dy, const void *x, const void *w_gate,
                                 const void *w_up, const void *w_down, const void *saved, void *dx, void *dw_gate,
                                 void *dw_up, void *dw_down, void *ws, void *stream)
{
    FfArgs a{};
    const conv2d_status_t st = check_ff(d, &a.z);
    if (st != CONV2D_OK) return st;
    if (!dw_gate || !dw_up || !dw_down) return CONV2D_ERR_NULL_POINTER;
    if (d->N > 0 && (!dy || !x || !w_gate || !w_up || !w_down || !saved || !dx)) return CONV2D_ERR_NULL_POINTER;
    const int64_t need = ff_bwd_ws_bytes(a.z);
    if (need < 0) return CONV2D_ERR_INVALID_DESC;
    if (!ws && need) return CONV2D_ERR_WORKSPACE;
    if (d->N > 0 && (!ff_inputs_aligned(a.z, x, w_gate, w_up, w_down) || !rows_aligned(dy, d->O, a.z.ldy, d->dtype)))
        return CONV2D_ERR_MISALIGNED;
    for (const void *p : {static_cast<const void *>(dx), static_cast<const void *>(dw_gate),
                          static_cast<const void *>(dw_up), static_cast<const void *>(dw_down)})
        if (!aligned(p, esize(d->dtype))) return CONV2D_ERR_MISALIGNED;
    if (!aligned(saved, 256) || !aligned(ws, 256)) return CONV2D_ERR_MISALIGNED;
    a.dy = dy;
    a.x = x;
    a.wg = w_gate;
    a.wu = w_up;
    a.wd = w_down;
    a.saved = const_cast<void *>(saved);
    a.dx = dx;
    a.dwg = dw_gate;
    a.dwu = dw_up;
    a.dwd = dw_down;
    a.ws = ws;
    return hip_status(launch_ff_bwd(a, static_cast<hipStream_t>(stream)));
}

conv2d_status_t residual_norm_fwd(const residual_norm_desc_t *d, const void *b, const void *r, const float *gate,
                                  const float *post_weight, const float *post_bias, const float *weight,
                                  const float *bias, void *out, void *y, float *stats, void *stream)
{
    ResNormArgs a;
    const conv2d_status_t st = check_res_norm(d, &a);
    if (st != CONV2D_OK) return st;
    if (!d->post && (post_weight || post_bias)) return CONV2D_ERR_INVALID_DESC;
    if (d->N == 0) return CONV2D_OK;
    if (!gate != !d->groups) return CONV2D_ERR_NULL_POINTER;
    if (!b || !r || !out || !y) return CONV2D_ERR_NULL_POINTER;
    if (!aligned(b, esize(d->branch_dtype)) || !aligned(y, esize(d->branch_dtype)) || !aligned(r, esize(d->dtype)) ||
        !aligned(out, esize(d->dtype)) || !aligned(stats, 16))
        return CONV2D_ERR_MISALIGNED;
    for (const float *p : {gate, post_weight, post_bias, weight, bias})
        if (!aligned(p, 4)) return CONV2D_ERR_MISALIGNED;
    a.b = b;
    a.r = r;
    a.gate = gate;
    a.pw = post_weight;
    a.pb = post_bias;
    a.w = weight;
    a.bias = bias;
    a.out = out;
    a.y = y;
    a.stats = stats;
    return hip_status(launch_res_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t residual_norm_bwd_workspace_size(const residual_norm_desc_t *d)
{
    ResNormArgs a;
    if (check_res_norm(d, &a) != CONV2D_OK) return 0;
    return size_t(res_norm_bwd_ws_bytes(d->N, d->C, d->groups));
}

conv2d_status_t residual_norm_bwd(const residual_norm_desc_t *d, const void *dy, const void *dout, const void *b,
                                  const void *out, const float *stats, const float *gate, const float *post_weight,
                                  const float *post_bias, const float *weight, void *dr, void *db, float *dgate,
                                  float *dpost_weight, float *dpost_bias, float *dweight, float *dbias, void *ws,
                                  void *stream)
{
    ResNormArgs a;
    const conv2d_status_t st = check_res_norm(d, &a);
    if (st != CONV2D_OK) return st;
    if (!d->post && (post_weight || post_bias || dpost_weight || dpost_bias)) return CONV2D_ERR_INVALID_DESC;
    if (dgate && !d->groups) return CONV2D_ERR_INVALID_DESC;
    const bool sums = dgate || dpost_weight || dpost_bias || dweight || dbias;
    if (d->N == 0 && !sums) return CONV2D_OK;
    if (d->N > 0 && (!gate != !d->groups || !dy || !b || !out || !stats || !dr || !db)) return CONV2D_ERR_NULL_POINTER;
    if (sums && !ws) return CONV2D_ERR_WORKSPACE;
    if (!aligned(dy, esize(d->branch_dtype)) || !aligned(b, esize(d->branch_dtype)) ||
        !aligned(db, esize(d->branch_dtype)) || !aligned(dout, esize(d->dtype)) || !aligned(out, esize(d->dtype)) ||
        !aligned(dr, esize(d->dtype)) || !aligned(stats, 16) || !aligned(ws, 256))
        return CONV2D_ERR_MISALIGNED;
    for (const float *p : {gate, post_weight, post_bias, weight, static_cast<const float *>(dgate),
                           static_cast<const float *>(dpost_weight), static_cast<const float *>(dpost_bias),
                           static_cast<const float *>(dweight), static_cast<const float *>(dbias)})
        if (!aligned(p, 4)) return CONV2D_ERR_MISALIGNED;
    a.dy = dy;
    a.dout = dout;
    a.b = b;
    a.out = const_cast<void *>(out);
    a.stats = const_cast<float *>(stats);
    a.gate = gate;
    a.pw = post_weight;
    a.pb = post_bias;
    a.w = weight;
    a.dr = dr;
    a.db = db;
    a.dgate = dgate;
    a.dpw = dpost_weight;
    a.dpb = dpost_bias;
    a.dw = dweight;
    a.dbias = dbias;
    a.ws = sums ? ws : nullptr;
    return hip_status(launch_res_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

conv2d_status_t adamw_step(const adamw_desc_t *d, const adamw_tensor_t *tensors, const int64_t *step_ptr,
                           const float *grad_scale_ptr, const float *lr_ptr, void *stream)
{
    if (!d) return CONV2D_ERR_NULL_POINTER;
    if (d->reserved != 0 || d->count < 0) return CONV2D_ERR_INVALID_DESC;
    if (d->bits != 32 && d->bits != 8) return CONV2D_ERR_UNSUPPORTED;
    if (!(d->beta1 >= 0.0 && d->beta1 < 1.0) || !(d->beta2 >= 0.0 && d->beta2 < 1.0)) return CONV2D_ERR_INVALID_DESC;
    if (!(d->eps >= 0.0) || !finite32(d->eps) || !finite32(d->grad_scale)) return CONV2D_ERR_INVALID_DESC;
    if (step_ptr ? d->step != 0 : d->step < 1) return CONV2D_ERR_INVALID_DESC;
    if (!aligned(step_ptr, 8) || !aligned(grad_scale_ptr, 4) || !aligned(lr_ptr, 4)) return CONV2D_ERR_MISALIGNED;
    if (d->count > 0 && !tensors) return CONV2D_ERR_NULL_POINTER;
    const bool coded = d->bits == 8;
    for (int64_t i = 0; i < d->count; ++i) {
        const adamw_tensor_t &t = tensors[i];
        if (t.reserved != 0 || t.n < 0 || t.n > kMaxElems) return CONV2D_ERR_INVALID_DESC;
        if (!type_ok(t.param_dtype) || !type_ok(t.grad_dtype) || (t.copy && !type_ok(t.copy_dtype)))
            return CONV2D_ERR_UNSUPPORTED;
        if (!finite32(t.lr) || !finite32(t.weight_decay)) return CONV2D_ERR_INVALID_DESC;
        if (coded ? t.first < 0 || t.first > int64_t(1) << 62 || t.first % 256 != 0 : t.first != 0)
            return CONV2D_ERR_INVALID_DESC;
        if (!coded && (t.m_scale || t.v_scale)) return CONV2D_ERR_INVALID_DESC;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (coded && (!t.m_scale || !t.v_scale)))
            return CONV2D_ERR_NULL_POINTER;
        if (!aligned(t.param, esize(t.param_dtype)) || !aligned(t.grad, esize(t.grad_dtype)) ||
            (t.copy && !aligned(t.copy, esize(t.copy_dtype))) || !aligned(t.m, 4) || !aligned(t.v, 4) ||
            !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
            return CONV2D_ERR_MISALIGNED;
    }
    AdamArgs a{};
    a.step_ptr = step_ptr;
    a.grad_scale_ptr = grad_scale_ptr;
    a.lr_ptr = lr_ptr;
    a.beta1 = d->beta1;
    a.beta2 = d->beta2;
    a.step = d->step;
    // 1 - beta^t without the cancellation of small steps (beta 0: 1)
    const auto correction = [&](double beta) { return beta > 0.0 ? -std::expm1(double(d->step) * std::log(beta)) : 1.0; };
    if (!step_ptr) {
        a.rate = 1.0 / correction(d->beta1);
        a.root = float(1.0 / std::sqrt(correction(d->beta2)));
    }
    a.seed = d->seed;
    a.eps = float(d->eps);
    a.grad_scale = float(d->grad_scale);
    int64_t chunks = 0;
    const auto launch = [&] {
        const hipError_t e = launch_adamw(a, d->bits, static_cast<hipStream_t>(stream));
        a.count = 0;
        chunks = 0;
        return hip_status(e);
    };
    // a launch has at most kAdamTensors tensors and kMost chunks; longer tensors are
    // taken in parts
    constexpr int64_t kMost = int64_t(1) << 22;
    const int64_t chunk = adam_chunk(d->bits);
    for (int64_t i = 0; i < d->count; ++i) {
        const adamw_tensor_t &t = tensors[i];
        for (int64_t at = 0; at < t.n;) {
            if (a.count == kAdamTensors || chunks == kMost) {
                const conv2d_status_t st = launch();
                if (st != CONV2D_OK) return st;
            }
            const int64_t n = std::min(t.n - at, (kMost - chunks) * chunk);
            chunks += (n + chunk - 1) / chunk;
            const auto part = [&](const void *p, int64_t size) {
                return p ? static_cast<char *>(const_cast<void *>(p)) + at * size : nullptr;
            };
            const int64_t ss = coded ? 1 : 4;
            a.t[a.count++] = AdamTensor{
                part(t.param, esize(t.param_dtype)), part(t.grad, esize(t.grad_dtype)), part(t.copy, esize(t.copy_dtype)),
                part(t.m, ss), part(t.v, ss), coded ? t.m_scale + at / 256 : nullptr, coded ? t.v_scale + at / 256 : nullptr,
                n, t.first + at, float(t.lr), float(t.weight_decay), int32_t(chunks), int8_t(t.param_dtype),
                int8_t(t.grad_dtype), int8_t(t.copy_dtype), 0};
            at += n;
        }
    }
    return a.count ? launch() : CONV2D_OK;
}

conv2d_status_t adamw_values(int64_t n, const void *m, const void *v, const float *m_scale, const float *v_scale,
                             float *m_values, float *v_values, void *stream)
{
    if (n < 0 || n > kMaxElems) return CONV2D_ERR_INVALID_DESC;
    if (n == 0) return CONV2D_OK;
    if (!m || !v || !m_scale || !v_scale || !m_values || !v_values) return CONV2D_ERR_NULL_POINTER;
    if (!aligned(m, 4) || !aligned(v, 4)) return CONV2D_ERR_MISALIGNED;
    for (const float *p : {m_scale, v_scale, static_cast<const float *>(m_values), static_cast<const float *>(v_values)})
        if (!aligned(p, 4)) return CONV2D_ERR_MISALIGNED;
    return hip_status(launch_adamw_values(n, m, v, m_scale, v_scale, m_values, v_values, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
