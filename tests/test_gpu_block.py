"""Block kernels (feed-forward block, norms around a residual sum, AdamW) against their
plain 64-bit forms (oracle/block.py), element by element.

Tolerances, derived from the operations as in test_gpu_head.py (u = 2^-24, uo the unit
roundoff of the stored type, sub half its smallest subnormal): a sum of n terms along
any chain is within 2 n u sum|terms| (twice n u, for matrix cores that truncate), every
other operation within a few u of its result, and an error e of an input passes through
a function of slope L as L e."""
import numpy as np
import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _block, _lib
from oracle import block as ref
from test_gpu_head import DEV, SUB, TYPES, U, UO, _close, _say

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.lib()


# ---- feed-forward block ----------------------------------------------------------------

# largest slopes of act and of act' (relu's jump at 0 is counted apart)
SLOPE = {"silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13, "relu": 1.0, "sigmoid": 0.25}
BEND = {"silu": 0.5, "gelu": 0.8, "gelu_tanh": 0.82, "relu": 0.0, "sigmoid": 0.1}


def _ff_case(N, D, F, O, dt, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device=DEV)
    t = TYPES[dt]
    return (rnd(N, D).to(t), (rnd(F, D) * 1.2 / D ** 0.5).to(t), (rnd(F, D) / D ** 0.5).to(t),
            (rnd(O, F) / F ** 0.5).to(t), (rnd(N, O) * scale).to(t))


def _ff_bounds(x, wg, wu, wd, dy, act, dt, few):
    """Bounds of (y, dx, dwg, dwu, dwd), and the exact ones."""
    N, D, F, O = x.shape[0], x.shape[1], wg.shape[0], wd.shape[0]
    X, G, W, Dn, DY = (v.double().abs() for v in (x, wg, wu, wd, dy))
    y, a, u, h = ref.feed_forward(x, wg, wu, wd, act)
    dx, dwg, dwu, dwd, da, du = ref.feed_forward_grad(dy, x, wg, wu, wd, act)
    uo = UO[dt] * 1.01 if dt != "f32" else 0.0
    ea, eu = 2 * (D + 1) * U * (X @ G.t()), 2 * (D + 1) * U * (X @ W.t())
    f, df = ref.activate(act, a)
    # expf, erff and their like: within (4 + |argument|) u of the result; half precision's
    # erfc within 1.5e-7, half of it in act / a and its slope
    more = (12 + 4 * a.abs()) * U * (1 + a.abs()) + (1e-7 * (1 + a.abs()) if act == "gelu" and dt != "f32" else 0.0)
    e1 = SLOPE[act] * ea + more                                     # of act(a)
    jump = (a.abs() <= ea).double() if act == "relu" else 0.0
    e2 = eu * df.abs() + u.abs() * (BEND[act] * ea + more + jump) + 2 * U * (u * df).abs()
    eh = e1 * u.abs() + f.abs() * eu + 2 * U * h.abs()
    ehr = eh + uo * h.abs() + (SUB[dt] if dt == "f16" else 0.0)
    # few rows: h in two parts, each rounded: uo^2 of it is left (fp16: or half a subnormal step)
    ehy = eh + uo * uo * h.abs() + (SUB[dt] if dt == "f16" else 0.0) if few else ehr
    last = UO[dt] * 1.01
    ty = ehy @ Dn.t() + 2 * (2 * F + 2) * U * (h.abs() @ Dn.t()) + last * y.abs() + SUB[dt]
    dh = dy.double() @ wd.double()
    edh = 2 * (O + 1) * U * (DY @ Dn)
    # fp16: held times S with S max|dy| >= 1/16, so half a subnormal step over S
    sub = SUB["f16"] * 16 * DY.max().item() if dt == "f16" else 0.0
    eda = edh * (u * df).abs() + dh.abs() * e2 + 2 * U * da.abs()
    edu = edh * f.abs() + dh.abs() * e1 + 2 * U * du.abs()
    eda, edu = eda + uo * (da.abs() + eda) + sub, edu + uo * (du.abs() + edu) + sub
    tx = eda @ G + edu @ W + 2 * (2 * F + 2) * U * (da.abs() @ G + du.abs() @ W) + last * dx.abs() + SUB[dt]
    tg = eda.t() @ X + 2 * (N + 2) * U * (da.abs().t() @ X) + last * dwg.abs() + SUB[dt]
    tu = edu.t() @ X + 2 * (N + 2) * U * (du.abs().t() @ X) + last * dwu.abs() + SUB[dt]
    td = DY.t() @ ehr + 2 * (N + 2) * U * (DY.t() @ h.abs()) + last * dwd.abs() + SUB[dt]
    return (ty, tx, tg, tu, td), (y, dx, dwg, dwu, dwd)


def _check_ff(case, act, dt, what="", save=True):
    x, wg, wu, wd, dy = case
    N, D, F, O = x.shape[0], x.shape[1], wg.shape[0], wd.shape[0]
    _say(f"feed-forward {what} N={N} D={D} F={F} O={O} {dt} {act}")
    few = N <= 16
    tol, want = _ff_bounds(x, wg, wu, wd, dy, act, dt, few)
    y, none = conv.feed_forward(x, wg, wu, wd, act, save=False)
    assert none is None
    _close(y, want[0], tol[0], "y")
    if not save:
        return
    y, saved = conv.feed_forward(x, wg, wu, wd, act)
    got = (y,) + conv.feed_forward_backward(dy, x, wg, wu, wd, saved, act)
    torch.cuda.synchronize()
    for g, w, t, name in zip(got, want, tol, ("y", "dx", "dw_gate", "dw_up", "dw_down")):
        _close(g, w, t, name)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", sorted(_block.ACTIVATIONS))
@pytest.mark.parametrize("N,D,F,O", [(1, 64, 96, 64), (16, 33, 47, 21), (17, 72, 200, 72), (65, 128, 256, 40)])
def test_feed_forward(N, D, F, O, act, dt):
    _check_ff(_ff_case(N, D, F, O, dt, seed=N + F), act, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,D,F,O", [
    (1, 1, 1, 1), (2, 1, 3, 1), (1, 7, 5, 2), (3, 9, 17, 8), (5, 1024, 16, 1000), (64, 31, 8, 24), (33, 40, 15, 16),
    (200, 8, 600, 8), (129, 136, 130, 264), (257, 264, 520, 128), (300, 100, 1000, 7), (1000, 24, 40, 32), (32, 256, 64, 512),
    (40, 500, 1031, 300), (15, 2050, 130, 33), (64, 65, 4097, 66)])
def test_feed_forward_sizes(N, D, F, O, dt):
    _check_ff(_ff_case(N, D, F, O, dt, seed=N + D), "silu", dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,D,F", [(4097, 264, 520), (2048, 1024, 1536), (700, 2048, 4104), (5000, 128, 300)])
def test_feed_forward_tiles(N, D, F, dt):
    """Sizes that take the larger tiles, split products, and the products in one launch."""
    _check_ff(_ff_case(N, D, F, D, dt, seed=N), "gelu", dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [5, 40, 150])
def test_feed_forward_strides_and_leading_dimensions(N, dt):
    """Views of wider tensors, strides of whole granules and not, starts off a granule
    where rows are copied anyway; x of more dimensions."""
    for D, F, O, pad, at in ((48, 72, 56, 16, 0), (48, 72, 56, 5, 0), (45, 70, 33, 4, 3)):
        x, wg, wu, wd, dy = _ff_case(N, D, F, O, dt, seed=pad)

        def wide(t):
            w = torch.full((t.shape[0], t.shape[1] + pad), NAN, dtype=t.dtype, device=DEV)
            w[:, at:at + t.shape[1]] = t
            return w[:, at:at + t.shape[1]]
        views = [wide(t) for t in (x, wg, wu, wd, dy)]
        _check_ff(views, "silu", dt, what=f"views +{pad} at {at}")
        y = wide(torch.zeros(N, O, dtype=x.dtype, device=DEV))
        ws = torch.empty(conv.feed_forward_workspace_size(*views[:4]) + 256, dtype=torch.uint8, device=DEV)
        conv.feed_forward_into(*views[:4], y, None, ws)
        assert torch.equal(y, conv.feed_forward(*views[:4], save=False)[0])
        assert bool(torch.isnan(y._base[:, at + O:]).all()), "outside y"
    x, wg, wu, wd, dy = _ff_case(24, 40, 64, 40, dt)
    y, saved = conv.feed_forward(x.view(2, 3, 4, 40), wg, wu, wd)
    y2, saved2 = conv.feed_forward(x, wg, wu, wd)
    assert y.shape == (2, 3, 4, 40) and torch.equal(y.view(24, 40), y2)
    got = conv.feed_forward_backward(dy.view(2, 3, 4, 40), x.view(2, 3, 4, 40), wg, wu, wd, saved)
    for a, b in zip(got, conv.feed_forward_backward(dy, x, wg, wu, wd, saved2)):
        assert torch.equal(a.reshape(b.shape), b)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 1e3])
def test_feed_forward_gradients_of_any_size(dt, scale):
    """fp16's da and du are scaled into range: gradients far from 1 keep their digits up to
    the outputs' own storage."""
    _check_ff(_ff_case(80, 96, 136, 64, dt, seed=5, scale=scale), "silu", dt, what=f"dy * {scale}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [9, 90])
def test_feed_forward_gradients_far_above_dy(N, dt):
    """da 10^5 times max |dy| (large Wu and Wd, a small gate) is finite in fp16 too."""
    x, wg, wu, wd, dy = _ff_case(N, 96, 136, 64, dt, seed=6, scale=1e-3)
    case = x, wg * 2.0 ** -4, wu * 512, wd * 256, dy
    da = ref.feed_forward_grad(dy, *case[:4], "silu")[4]
    assert da.abs().max().item() > 65504 * dy.abs().max().item()
    _check_ff(case, "silu", dt)


def test_feed_forward_no_rows():
    for dt in TYPES.values():
        x, w, wd = torch.empty(0, 8, dtype=dt, device=DEV), torch.ones(5, 8, dtype=dt, device=DEV), torch.ones(
            3, 5, dtype=dt, device=DEV)
        y, saved = conv.feed_forward(x, w, w, wd)
        assert y.shape == (0, 3)
        dx, *dw = conv.feed_forward_backward(y, x, w, w, wd, saved)
        assert dx.shape == (0, 8) and not any(bool(g.any()) for g in dw)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [3, 70])
def test_feed_forward_rows_by_themselves(N, dt):
    """NaN and infinities of one row of x stay in its row of y and dx; rows whose dy is 0
    (padding) add nothing to the weights' gradients whatever finite values x holds."""
    x, wg, wu, wd, dy = _ff_case(N, 40, 72, 24, dt, seed=2)
    y0, s0 = conv.feed_forward(x, wg, wu, wd)
    dx0 = conv.feed_forward_backward(dy, x, wg, wu, wd, s0)[0]
    rest = torch.arange(N, device=DEV) != 1
    for value in (NAN, INF):
        bad = x.clone()
        bad[1, 3] = value
        y, s = conv.feed_forward(bad, wg, wu, wd)
        dx = conv.feed_forward_backward(dy, bad, wg, wu, wd, s)[0]
        assert torch.equal(y[rest], y0[rest]) and torch.equal(dx[rest], dx0[rest])
        assert not bool(torch.isfinite(y[1]).any())
    dy[1] = 0
    want = conv.feed_forward_backward(dy, x, wg, wu, wd, s0)[1:]
    bad = x.clone()
    bad[1] = 100.0
    _, s = conv.feed_forward(bad, wg, wu, wd)
    for a, b in zip(conv.feed_forward_backward(dy, bad, wg, wu, wd, s)[1:], want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,D,F", [(7, 33, 50), (130, 100, 700), (600, 256, 1024), (300, 40, 90)])
def test_feed_forward_reads_nothing_it_has_not_written(N, D, F, dt):
    """Workspaces and saved buffers full of NaN bytes and of zeros give the same bits; a
    buffer behind each one's size is left as it was."""
    x, wg, wu, wd, dy = _ff_case(N, D, F, D, dt, seed=1)
    nw = conv.feed_forward_workspace_size(x, wg, wu, wd, saved=True, dy=dy)
    ns, n0 = conv.feed_forward_saved_size(x, wg), conv.feed_forward_workspace_size(x, wg, wu, wd)
    outs = []
    for fill in (0, 255):
        ws, sv = (torch.full((n + 64,), fill, dtype=torch.uint8, device=DEV) for n in (max(nw, n0), ns))
        y, y1 = torch.empty_like(dy), torch.empty_like(dy)
        g = [torch.empty_like(t) for t in (x, wg, wu, wd)]
        conv.feed_forward_into(x, wg, wu, wd, y1, None, ws)
        ws.fill_(fill)
        conv.feed_forward_into(x, wg, wu, wd, y, sv, ws)
        ws.fill_(fill)
        conv.feed_forward_backward_into(dy, x, wg, wu, wd, sv, *g, ws)
        assert bool((ws[max(nw, n0):] == fill).all()) and bool((sv[ns:] == fill).all())
        outs.append([y1, y] + g)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("N,D,F,O,dt", [
    (1, 40, 16384, 24, "bf16"), (5, 24, 2500, 40, "f16"), (16, 512, 4096, 1024, "bf16"), (33, 72, 1600, 72, "f32"),
    (48, 33, 3001, 201, "f16"), (64, 520, 8200, 300, "f32"), (24, 2048, 8192, 640, "f32"), (40, 129, 9001, 100, "f16")])
def test_feed_forward_few_rows_and_outputs(N, D, F, O, dt):
    """y's sum over the hidden features split over workgroups: its bound; the same bits from
    every run, replayed ones among them, whatever the workspace holds."""
    x, wg, wu, wd, dy = case = _ff_case(N, D, F, O, dt, seed=N + F)
    _check_ff(case, "silu", dt)
    n = conv.feed_forward_workspace_size(x, wg, wu, wd)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=DEV)
    y, want = torch.empty_like(dy), conv.feed_forward(x, wg, wu, wd, save=False)[0]
    for fill in (255, 0, 1):
        ws.fill_(fill)
        for _ in range(4):
            y.fill_(NAN)
            conv.feed_forward_into(x, wg, wu, wd, y, None, ws)
            assert torch.equal(y, want)
        assert bool((ws[n:] == fill).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        conv.feed_forward_into(x, wg, wu, wd, y, None, ws)
    for _ in range(3):
        y.fill_(NAN)
        ws.fill_(255)
        graph.replay()
        assert torch.equal(y, want)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "sigmoid"])
def test_feed_forward_gradients_against_differences(act):
    x, wg, wu, wd, dy = _ff_case(30, 48, 80, 40, "f32", seed=9)
    g = torch.Generator(device=DEV).manual_seed(1)
    e = [torch.randn(t.shape, generator=g, device=DEV) * 0.1 for t in (x, wg, wu, wd)]

    def f(h):
        y, _ = conv.feed_forward(*(t + h * d for t, d in zip((x, wg, wu, wd), e)), act, save=False)
        return (y.double() * dy.double()).sum().item()
    _, saved = conv.feed_forward(x, wg, wu, wd, act)
    grads = conv.feed_forward_backward(dy, x, wg, wu, wd, saved, act)
    want = sum((a.double() * d.double()).sum().item() for a, d in zip(grads, e))
    h = 2.0 ** -5
    # fourth-order differences: sums of 1200 terms of order 1 with error 2^-20 over 2h
    got = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
    assert abs(got - want) <= 2e-3 * max(1.0, sum(a.double().norm().item() * 0.1 for a in grads)), (got, want)


# ---- norms around a residual sum ----------------------------------------------------------

def _rn_case(N, C, G, rt, bt, post, seed=0, affine=True):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=g, device=DEV)
    lev = rnd(1, C)
    c = dict(b=(rnd(N, C) * 1.5 + lev).to(TYPES[bt]), r=(2 * rnd(N, C) + lev).to(TYPES[rt]),
             gate=0.5 + 0.3 * rnd(G, C) if G else None, dy=rnd(N, C).to(TYPES[bt]), dout=rnd(N, C).to(TYPES[rt]))
    c["w"], c["bias"] = (1 + 0.3 * rnd(C), 0.5 * rnd(C)) if affine else (None, None)
    c["pw"], c["pb"] = (1 + 0.3 * rnd(C), 0.5 * rnd(C)) if affine and post else (None, None)
    return c


def _ones(v, value, like):
    return torch.full((1,), value, dtype=torch.float64, device=like.device) if v is None else v.double()


def _norm_error(z, ez, mean, rstd, kind, eps, D1):
    """(of the mean, relative of rstd) for a row z with elementwise errors ez."""
    dm = ez.mean(1, keepdim=True) + D1 * U * z.abs().mean(1, keepdim=True) + U * mean.abs() if kind == "layer" else \
        torch.zeros_like(mean)
    d = z - mean
    dv = (2 * d.abs() * (ez + dm) + (ez + dm) ** 2).mean(1, keepdim=True)
    return dm, 0.5 * (dv * rstd ** 2 + (D1 + 4) * U) + 4 * U


def _check_rn(c, rt, bt, kind, post, rs=0.9, bs=1.1, eps=1e-5, dout=True, what=""):
    b, r = c["b"], c["r"]
    N, C = b.shape
    G = 0 if c["gate"] is None else c["gate"].reshape(-1, C).shape[0]
    _say(f"residual norm {what} {N}x{C} gates {G} {rt}/{bt} {kind} post={post}")
    kw = dict(gate=c["gate"], post_weight=c["pw"], weight=c["w"], kind=kind, post=post, residual_scale=rs, branch_scale=bs)
    out, y, st = conv.residual_norm(b, r, eps, post_bias=c["pb"], bias=c["bias"], **kw)
    torch.cuda.synchronize()
    o0, y0, s0, p0 = ref.residual_norm(b, r, c["gate"], c["pw"], c["pb"], c["w"], c["bias"], kind, post, eps, rs, bs)
    D1, D2 = C / 32 + 64, N / 64 + 256
    g = ref.row_gates(c["gate"], N, b)
    pw, pb, w, bias = _ones(c["pw"], 1, b), _ones(c["pb"], 0, b), _ones(c["w"], 1, b), _ones(c["bias"], 0, b)
    B, R = b.double(), r.double()
    m1, r1, m2, r2 = (v[:, None] for v in s0.unbind(1))
    tp = torch.zeros_like(B)
    if post:
        dm, rho = _norm_error(B, torch.zeros_like(B), m1, r1, kind, eps, D1)
        _close(st[:, 0:1], m1, dm + 2 * U * m1.abs() + 1e-300, "mean of the branch")
        _close(st[:, 1:2], r1, rho * r1, "rstd of the branch")
        h = (B - m1) * r1
        tp = pw.abs() * r1 * dm + (h * pw).abs() * (rho + 6 * U) + 4 * U * (p0.abs() + pb.abs())
    else:
        assert not st[:, :2].any()
    to = (bs * g).abs() * tp + 5 * U * ((rs * R).abs() + (bs * g * p0).abs())
    _close(out, o0, to + UO[rt] * 1.01 * o0.abs() + SUB[rt], "out")
    dm, rho = _norm_error(o0, to, m2, r2, kind, eps, D1)
    _close(st[:, 2:3], m2, dm + 2 * U * m2.abs() + 1e-300, "mean of out")
    _close(st[:, 3:4], r2, rho * r2, "rstd of out")
    h = (o0 - m2) * r2
    ty = w.abs() * r2 * (to + dm) + (h * w).abs() * (rho + 6 * U) + 4 * U * (y0.abs() + bias.abs())
    _close(y, y0, ty + UO[bt] * 1.01 * y0.abs() + SUB[bt], "y")

    do = c["dout"] if dout else None
    dr, db, grads = conv.residual_norm_backward(c["dy"], do, b, out, st, post_bias=c["pb"], **kw)
    torch.cuda.synchronize()
    q = ref.residual_norm_grad(c["dy"], do, b, out, st, c["gate"], c["pw"], c["pb"], c["w"], kind, post, rs, bs)
    m1, r1, m2, r2 = (v[:, None] for v in st.double().unbind(1))
    DY, DO = c["dy"].double(), (do.double() if dout else torch.zeros_like(B))
    h = (out.double() - m2) * r2
    z = DY * w
    lay = 1.0 if kind == "layer" else 0.0
    e1 = lay * (D1 + 5) * U * z.abs().mean(1, keepdim=True)
    e2 = (D1 + 8) * U * (z * h).abs().mean(1, keepdim=True)
    sums = z.abs() + lay * z.mean(1, keepdim=True).abs() + (h * (z * h).mean(1, keepdim=True)).abs()
    tt = r2 * (e1 + h.abs() * e2 + 8 * U * sums) + 3 * U * q["t"].abs() + 2 * U * DO.abs()
    _close(dr, q["dr"], abs(rs) * tt + (U + UO[rt] * 1.01) * q["dr"].abs() + SUB[rt], "dr")
    _close(grads["weight"], q["weight"], (D2 + 8) * U * (DY * h).abs().sum(0) + 1e-30, "dweight")
    _close(grads["bias"], q["bias"], (D2 + 4) * U * DY.abs().sum(0) + 1e-30, "dbias")
    gq = (bs * g).abs()
    if post:
        k = (B - m1) * r1
        t = q["t"].abs()
        _close(grads["post_weight"], q["post_weight"],
               (gq * (tt * k.abs() + (D2 + 12) * U * t * k.abs())).sum(0) + 1e-30, "dpost_weight")
        _close(grads["post_bias"], q["post_bias"], (gq * (tt + (D2 + 12) * U * t)).sum(0) + 1e-30, "dpost_bias")
        v = bs * g * q["t"] * pw
        tv = (gq * pw.abs()) * tt + 4 * U * v.abs()
        e3 = lay * (tv.mean(1, keepdim=True) + (D1 + 5) * U * v.abs().mean(1, keepdim=True))
        e4 = (tv * k.abs()).mean(1, keepdim=True) + (D1 + 8) * U * (v * k).abs().mean(1, keepdim=True)
        sums = v.abs() + lay * v.mean(1, keepdim=True).abs() + (k * (v * k).mean(1, keepdim=True)).abs()
        tb = r1 * (tv + e3 + k.abs() * e4 + 8 * U * sums)
        share = abs(bs) * (tt * ((k * pw).abs() + pb.abs()) + (D2 + 16) * U * t * ((k * pw).abs() + pb.abs()))
    else:
        tb = gq * tt + 4 * U * q["db"].abs()
        share = abs(bs) * (tt + (D2 + 16) * U * q["t"].abs()) * B.abs()
        assert "post_weight" not in grads
    _close(db, q["db"], tb + UO[bt] * 1.01 * q["db"].abs() + SUB[bt], "db")
    if G:
        _close(grads["gate"].reshape(G, C), q["gate"], share.reshape(G, N // G, C).sum(1) + 1e-30, "dgate")
    return out, y, st, dr, db, grads


TYPE_PAIRS = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]


@pytest.mark.parametrize("rt,bt", TYPE_PAIRS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("N,C,G", [(1, 512, 1), (5, 1, 0), (7, 5, 7), (40, 8, 4), (33, 65, 3), (300, 130, 1), (65, 1001, 5),
                                   (24, 2047, 0), (30, 4096, 3), (9, 6001, 9), (12, 8200, 2)])
def test_residual_norm(N, C, G, kind, post, rt, bt):
    _check_rn(_rn_case(N, C, G, rt, bt, post, seed=N + C), rt, bt, kind, post)


@pytest.mark.parametrize("rt,bt", [("f32", "f32"), ("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("N,C,G", [(70000, 4, 1), (1001, 7, 91), (4096, 2, 4096), (2500, 3, 50), (600, 1, 2), (513, 6, 0),
                                   (130000, 5, 13)])
def test_residual_norm_of_short_rows(N, C, G, rt, bt):
    """Rows of fewer channels than a vector has: a lane to each."""
    # (one channel's deviation from its mean is 0 or what is lost of it: RMS norms for it)
    _check_rn(_rn_case(N, C, G, rt, bt, True, seed=C), rt, bt, "rms" if C == 1 else "layer", True)


@pytest.mark.parametrize("rt,bt", [("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("N,C,G", [(5000, 64, 50), (20000, 256, 1), (4096, 1000, 4096), (3000, 520, 1000), (777, 24, 777),
                                   (2310, 96, 7), (1024, 3000, 3), (600, 9000, 60), (40960, 64, 4096), (1300, 6000, 325),
                                   (9000, 1001, 600), (60000, 3, 6000)])
def test_residual_norm_of_many_rows_and_gates(N, C, G, rt, bt):
    if N % max(G, 1):
        N = N // G * G
    _check_rn(_rn_case(N, C, G, rt, bt, True, seed=C), rt, bt, "layer", True)


@pytest.mark.parametrize("C", [33, 512, 9001])
def test_residual_norm_without_parameters_or_gradients(C):
    for kind in ("layer", "rms"):
        c = _rn_case(20, C, 0, "f32", "bf16", True, affine=False)
        out, y, st, dr, db, _ = _check_rn(c, "f32", "bf16", kind, True, dout=False)
        a, d = torch.empty_like(dr), torch.empty_like(db)
        conv.residual_norm_backward_into(c["dy"], None, c["b"], out, st, a, d, None, kind=kind, residual_scale=0.9,
                                         branch_scale=1.1)
        assert torch.equal(a, dr) and torch.equal(d, db)
        o2, y2 = torch.empty_like(out), torch.empty_like(y)
        conv.residual_norm_into(c["b"], c["r"], o2, y2, None, kind=kind, residual_scale=0.9, branch_scale=1.1)
        assert torch.equal(o2, out) and torch.equal(y2, y)


@pytest.mark.parametrize("some", ["gate", "post_weight", "post_bias", "weight", "bias"])
@pytest.mark.parametrize("N,C", [(30, 100), (330, 100), (30, 9001), (500, 5)])
def test_residual_norm_single_gradients(some, N, C):
    c = _rn_case(N, C, 5, "f32", "f32", True)
    kw = dict(gate=c["gate"], post_weight=c["pw"], post_bias=c["pb"], weight=c["w"])
    out, _, st = conv.residual_norm(c["b"], c["r"], bias=c["bias"], **kw)
    dr, db, want = conv.residual_norm_backward(c["dy"], c["dout"], c["b"], out, st, **kw)
    g = torch.empty_like(want[some])
    ws = torch.full((conv.residual_norm_workspace_size(c["b"], gate=c["gate"]),), 255, dtype=torch.uint8, device=DEV)
    conv.residual_norm_backward_into(c["dy"], c["dout"], c["b"], out, st, torch.empty_like(dr), torch.empty_like(db), ws,
                                     **kw, **{"d" + some: g})
    assert torch.equal(g, want[some])


@pytest.mark.parametrize("C", [40, 300, 8201])
def test_residual_norm_strides(C):
    """Rows of one stride of wider tensors; what lies between them stays."""
    c = _rn_case(14, C, 7, "f32", "f16", True)

    def wide(t, pad=11):
        w = torch.full((t.shape[0], C + 3 + pad), 7.0, dtype=t.dtype, device=DEV)
        w[:, 3:3 + C] = t
        return w[:, 3:3 + C]
    kw = dict(gate=c["gate"], post_weight=c["pw"], post_bias=c["pb"], weight=c["w"])
    out, y, st = conv.residual_norm(c["b"], c["r"], bias=c["bias"], **kw)
    dr, db, grads = conv.residual_norm_backward(c["dy"], c["dout"], c["b"], out, st, **kw)
    b, r, o, yy = wide(c["b"]), wide(c["r"], 2), wide(out * 0, 5), wide(y * 0, 8)
    st2 = torch.empty_like(st)
    conv.residual_norm_into(b, r, o, yy, st2, bias=c["bias"], **kw)
    assert torch.equal(o, out) and torch.equal(yy, y) and torch.equal(st2, st)
    a, d = wide(dr * 0, 4), wide(db * 0, 9)
    g = {"d" + k: torch.empty_like(v) for k, v in grads.items()}
    ws = torch.empty(conv.residual_norm_workspace_size(b, gate=c["gate"], residual_dtype=torch.float32), dtype=torch.uint8,
                     device=DEV)
    conv.residual_norm_backward_into(wide(c["dy"]), wide(c["dout"], 1), b, o, st2, a, d, ws, **kw, **g)
    assert torch.equal(a, dr) and torch.equal(d, db) and all(torch.equal(g["d" + k], v) for k, v in grads.items())
    for t in (o, yy, a, d):
        assert bool((t._base[:, :3] == 7).all()) and bool((t._base[:, 3 + C:] == 7).all())


def test_residual_norm_no_rows():
    b = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV)
    gate = torch.ones(3, 24, device=DEV)
    out, y, st = conv.residual_norm(b, b, gate=gate)
    dr, db, grads = conv.residual_norm_backward(y, out, b, out, st, gate=gate)
    assert out.shape == (0, 24) and st.shape == (0, 4) and dr.shape == (0, 24)
    assert grads["gate"].shape == (3, 24) and not any(bool(g.any()) for g in grads.values())


@pytest.mark.parametrize("C", [64, 700, 4096, 9000])
def test_residual_norm_rows_by_themselves(C):
    """NaN and infinities of one row reach that row alone; a row of zeros has eps alone."""
    c = _rn_case(20, C, 1, "f32", "bf16", True)
    rest = torch.arange(20, device=DEV) != 4
    kw = dict(gate=c["gate"], weight=c["w"])
    o0, y0, s0 = conv.residual_norm(c["b"], c["r"], **kw)
    for value in (NAN, INF):
        b = c["b"].clone()
        b[4, C // 2] = value
        out, y, st = conv.residual_norm(b, c["r"], **kw)
        assert all(torch.equal(p[rest], q[rest]) for p, q in ((out, o0), (y, y0), (st, s0)))
        assert bool(torch.isnan(y[4]).all())
    z = torch.zeros(2, C, device=DEV)
    for kind in ("layer", "rms"):
        out, y, st = conv.residual_norm(z, z, kind=kind)
        assert not out.any() and not y.any()
        assert bool(((st - torch.tensor([0, 1e-5 ** -0.5, 0, 1e-5 ** -0.5], device=DEV)).abs() <= 4 * U * 317).all())


# ---- AdamW ---------------------------------------------------------------------------------

def _adam_case(sizes, pt, gt, bits, seed=0, t=7):
    g = torch.Generator().manual_seed(seed)
    params = [(0.1 * torch.randn(n, generator=g)).to(TYPES[pt]) for n in sizes]
    grads = [(torch.randn(n, generator=g) * 10 ** (k % 5 - 3)).to(TYPES[gt]) for k, n in enumerate(sizes)]
    for q in grads:
        q[::7] = 0
    state = conv.adamw_state([p.to(DEV) for p in params], bits)
    ms, vs = [], []
    for k, (n, at) in enumerate(zip(state.sizes, state.first)):
        m = 0.3 * torch.randn(n, generator=g, dtype=torch.float64) * 10.0 ** (k % 5 - 3)
        v = (torch.randn(n, generator=g, dtype=torch.float64) * 10.0 ** (k % 5 - 3)) ** 2
        m[::5], v[::5] = 0, 0
        if bits == 8 and n:
            mk, vk, s, z = ref.encode(m, v, at, t - 1, 5)
            nb = s.numel()
            state.exp_avg[at:at + n], state.exp_avg_sq[at:at + n] = mk.to(DEV), vk.to(DEV)
            state.exp_avg_scale[at // 256:at // 256 + nb] = s.to(DEV)
            state.exp_avg_sq_scale[at // 256:at // 256 + nb] = z.to(DEV)
            m, v = ref.decode(mk, vk, s, z)
        elif n:
            m, v = m.float().double(), v.float().double()
            state.exp_avg[at:at + n], state.exp_avg_sq[at:at + n] = m.float().to(DEV), v.float().to(DEV)
        ms.append(m)
        vs.append(v)
    return params, grads, state, ms, vs


def _scales(state, k):
    """Tensor k's scales of m and of v."""
    a = state.first[k] // 256
    b = a + -(-state.sizes[k] // 256)
    return state.exp_avg_scale[a:b].cpu(), state.exp_avg_sq_scale[a:b].cpu()


HYPER = dict(beta1=0.9, beta2=0.999, eps=1e-8)


def _check_adam(sizes, pt, gt, bits, ct=None, t=7, seed=0, lr=1e-2, decay=0.1, gs=0.5):
    _say(f"adamw {len(sizes)} tensors {sizes[:4]} {pt}/{gt}/{ct} {bits} bits step {t}")
    params, grads, state, ms, vs = _adam_case(sizes, pt, gt, bits, seed, t)
    pd, gd = [p.to(DEV) for p in params], [q.to(DEV) for q in grads]
    cd = None if ct is None else [torch.empty(n, dtype=TYPES[ct], device=DEV) if k % 3 != 1 else None
                                  for k, n in enumerate(sizes)]
    rates = [lr * (1 + k % 3) for k in range(len(sizes))]
    decays = [decay * (k % 2) for k in range(len(sizes))]
    conv.adamw(pd, gd, state, t, rates, weight_decay=decays, grad_scale=gs, copies=cd, seed=77, **HYPER)
    torch.cuda.synchronize()
    for k, (n, at) in enumerate(zip(state.sizes, state.first)):
        g = (grads[k].float() * gs).double()
        want, m, v = ref.adamw(params[k], g, ms[k], vs[k], t, rates[k], 0.9, 0.999, 1e-8, decays[k])
        em = 4 * U * (0.9 * ms[k].abs() + 0.1 * g.abs()) + 2.0 ** -149
        ev = 6 * U * v + 2.0 ** -149
        if bits == 32:
            _close(state.exp_avg[at:at + n], m, em, "m")
            _close(state.exp_avg_sq[at:at + n], v, ev, "v")
        else:
            if n == 0:
                continue
            mk, vk, _, _ = ref.encode(m, v, at, t, 77, _scales(state, k))
            assert torch.equal(state.exp_avg[at:at + n].cpu(), mk), "m codes"
            assert torch.equal(state.exp_avg_sq[at:at + n].cpu(), vk), "v codes"
        # the update's relative error: m, sqrt(v), their factors, a root and a quotient
        upd = (params[k].double() * (1 - rates[k] * decays[k]) - want).abs()
        den = torch.sqrt(v / (1 - 0.999 ** t)) + 1e-8
        tol = rates[k] / (1 - 0.9 ** t) * em / den + 24 * U * upd + 4 * U * params[k].double().abs()
        _close(pd[k], want, tol + UO[pt] * 1.01 * want.abs() + SUB[pt], "p")
        if cd is not None and cd[k] is not None:
            _close(cd[k], want, tol + UO[ct] * 1.01 * want.abs() + SUB[ct], "copy")
    if bits == 8:
        mv, vv = conv.adamw_state_values(state)
        m0, v0 = ref.decode(state.exp_avg.cpu(), state.exp_avg_sq.cpu(), state.exp_avg_scale.cpu(),
                            state.exp_avg_sq_scale.cpu())
        _close(mv, m0, U * 1.01 * m0.abs() + 2.0 ** -149, "values of m")
        _close(vv, v0, U * 1.01 * v0.abs() + 2.0 ** -149, "values of v")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gt", ["f32", "f16", "bf16"])
def test_adamw(pt, gt, bits):
    _check_adam([1, 3, 255, 256, 257, 1023, 1024, 1025, 2049, 5000], pt, gt, bits, ct="bf16" if pt == "f32" else None)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0, 700], [20000], [37 * k + 1 for k in range(95)]])
@pytest.mark.parametrize("t", [1, 1000, 1 << 33])
def test_adamw_tensors_and_steps(sizes, t, bits):
    if t > 1 and len(sizes) > 50:
        sizes = sizes[:3]
    _check_adam(sizes, "f32", "bf16", bits, ct="f16", t=t, seed=3)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_views_and_steps_one_after_another(bits):
    """Tensors at odd places of a flat buffer; 30 steps as the definition takes them."""
    sizes = [5, 301, 1, 2050, 777]
    g = torch.Generator().manual_seed(1)
    flat = 0.1 * torch.randn(sum(sizes), generator=g)
    fd = flat.to(DEV)
    params = list(fd.split(sizes))
    state = conv.adamw_state(params, bits)
    p = [v.double() for v in flat.split(sizes)]
    m = [torch.zeros(n, dtype=torch.float64) for n in sizes]
    v = [torch.zeros(n, dtype=torch.float64) for n in sizes]
    for t in range(1, 31):
        grad = torch.randn(sum(sizes), generator=g)
        conv.adamw(params, list(grad.to(DEV).split(sizes)), state, t, 1e-3, weight_decay=0.01, seed=4)
        for k, q in enumerate(grad.split(sizes)):
            p[k], m[k], v[k] = ref.adamw(p[k], q, m[k], v[k], t, 1e-3, 0.9, 0.999, 1e-8, 0.01)
            if bits == 8:
                m[k], v[k] = ref.decode(*ref.encode(m[k], v[k], state.first[k], t, 4, _scales(state, k)))
    for k, q in enumerate(params):
        # 30 updates of at most about 3e-3 (|m / sqrt(v)| < 3.2 with these betas), 32 roundings of each
        _close(q, p[k], torch.tensor(30 * (4 * U * 0.6 + 32 * U * 3.2e-3)), f"tensor {k}")
        n, at = sizes[k], state.first[k]
        got = conv.adamw_state_values(state)[0][at:at + n]
        _close(got, m[k], 31 * 4 * U * torch.tensor(4.0) if bits == 32 else U * 1.01 * m[k].abs() + 2.0 ** -149, "m")


def test_adamw_8_bit_blocks_without_finite_values():
    """NaN or infinity in a block's gradient: its scales are NaN, its parameters' own step is
    that of fp32, and no other block sees it. Blocks of zeros stay zeros."""
    n = 256 * 4
    p = torch.ones(n, device=DEV)
    for value in (NAN, INF, -INF):
        g = torch.full((n,), 0.5, device=DEV)
        g[300] = value
        g[512:768] = 0
        state = conv.adamw_state([p], 8)
        q = p.clone()
        conv.adamw([q], [g], state, 1, 0.1)
        s = state.exp_avg_scale.cpu(), state.exp_avg_sq_scale.cpu()
        for t in s:
            assert torch.isnan(t[1]) and bool(torch.isfinite(t[[0, 2, 3]]).all()) and t[2] == 0
        assert not state.exp_avg[256:768].any() and not state.exp_avg_sq[256:768].any()
        keep = torch.ones(n, dtype=torch.bool, device=DEV)
        keep[300] = False
        assert bool(torch.isfinite(q[keep]).all()) and bool((q[512:768] == 1).all())


def test_adamw_8_bit_v_never_leaves_an_element_without_a_denominator():
    """Elements a millionth of their block's largest keep v > 0: their step stays bounded."""
    g = torch.full((256,), 1e-6, device=DEV)
    g[0] = 1.0
    p = torch.zeros(256, device=DEV)
    state = conv.adamw_state([p], 8)
    for t in range(1, 50):
        conv.adamw([p], [g], state, t, 1e-3, seed=t)
        assert bool((state.exp_avg_sq >= 1).all())
    # |m / sqrt(v)| of a constant gradient is 1, quantised m at most 2 levels of 1 / 127^2, sqrt(v) at least 1 / 255^2
    assert bool((p.abs() <= 49 * 1e-3 * 8).all())


def test_adamw_device_scalars():
    """The step, the gradients' scale and the rates' scale from device memory."""
    for bits in (32, 8):
        a, b = (_adam_case([300, 2000], "f32", "bf16", bits, seed=2) for _ in range(2))
        outs = []
        for (params, grads, state, _, _), scalars in ((a, False), (b, True)):
            pd, gd = [p.to(DEV) for p in params], [q.to(DEV) for q in grads]
            one = lambda v, t=torch.float32: torch.tensor([v], dtype=t, device=DEV)   # noqa: E731
            if scalars:
                conv.adamw(pd, gd, state, one(7, torch.int64), 1e-2, weight_decay=0.1, grad_scale=one(0.25), seed=3,
                           lr_scale=one(0.5))
            else:
                conv.adamw(pd, gd, state, 7, 0.5e-2, weight_decay=0.1, grad_scale=0.25, seed=3)
            outs.append(pd + [state.exp_avg, state.exp_avg_sq])
        for x, y in zip(*outs):
            if x.dtype is torch.float32:
                # 1 - beta^t by another route, lr times a half: two roundings of the update
                assert bool(((x - y).abs() <= 4 * U * (x.abs() + 0.1)).all())
            else:
                assert torch.equal(x, y)


# ---- more than 2^32 elements ------------------------------------------------------------------

def _half(seed, dt, *shape, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(shape, dtype=TYPES[dt], device=DEV)
    for part in t.split(1 << 16):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * scale)
    return t


def test_residual_norm_beyond_32_bits():
    """Rows before, across and past 2^31 and 2^32 elements are what they are by themselves."""
    N, C = (1 << 20) + 3, 4100
    b, r, dy, dout = (_half(k, "bf16", N, C) for k in range(4))
    w = torch.linspace(0.5, 2.0, C, device=DEV)
    out, y, st = conv.residual_norm(b, r, weight=w, post_weight=w)
    dr, db, grads = conv.residual_norm_backward(dy, dout, b, out, st, weight=w, post_weight=w)
    for at in (0, (1 << 31) // C - 5, (1 << 32) // C - 9, N - 12):
        part = slice(at, at + 12)
        b1, r1, dy1, do1 = (t[part].clone() for t in (b, r, dy, dout))
        o1, y1, s1 = conv.residual_norm(b1, r1, weight=w, post_weight=w)
        dr1, db1, _ = conv.residual_norm_backward(dy1, do1, b1, o1, s1, weight=w, post_weight=w)
        for name, t, t1 in (("out", out, o1), ("y", y, y1), ("stats", st, s1), ("dr", dr, dr1), ("db", db, db1)):
            assert torch.equal(t[part], t1), (name, at)
    want, size = (torch.zeros(C, dtype=torch.float64, device=DEV) for _ in range(2))
    for part in dy.split(1 << 16):
        want += part.double().sum(0)
        size += part.double().abs().sum(0)
    # 4097 rows a workgroup one after another, 256 workgroups in a tree
    _close(grads["bias"], want, 4200 * U * size, "dbias")
    del b, r, dy, dout, out, y, st, dr, db, part, b1, r1, dy1, do1
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,D,F,O,dt", [(3, 4104, 1 << 20, 40, "bf16"), (40, 4103, (1 << 20) - 1, 24, "f16"),
                                        (130, 40, 1 << 20, 4104, "bf16")])
def test_feed_forward_beyond_32_bits(N, D, F, O, dt):
    """Weights and their gradients of more than 2^32 elements: features at both ends and in
    the middle against the formulas, the others' share of y and dx by zeros in Wd."""
    x, wg, wu = _half(1, dt, N, D), _half(2, dt, F, D, scale=D ** -0.5), _half(3, dt, F, D, scale=D ** -0.5)
    dy, wd = _half(4, dt, N, O), torch.zeros(O, F, dtype=TYPES[dt], device=DEV)
    some = torch.tensor([0, 1, 17, F // 2 - 1, F // 2 + 3, F - 18, F - 2, F - 1], device=DEV)
    wd[:, some] = _half(5, dt, O, len(some))
    y, saved = conv.feed_forward(x, wg, wu, wd)
    got = (y,) + conv.feed_forward_backward(dy, x, wg, wu, wd, saved)
    tol, want = _ff_bounds(x, wg[some], wu[some], wd[:, some].contiguous(), dy, "silu", dt, N <= 16)
    # (the bounds' sums are over the features that count: the zeros add none)
    for g, w, t, name in zip((got[0], got[1], got[2][some], got[3][some], got[4][:, some]), want, tol,
                             ("y", "dx", "dw_gate", "dw_up", "dw_down")):
        _close(g, w, t, name)
    rest = torch.tensor([2, F // 3, F - 3], device=DEV)
    assert not bool(got[2][rest].any()) and not bool(got[3][rest].any())
    del x, wg, wu, wd, dy, y, saved, got, g
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_beyond_32_bits(bits):
    n, last = (1 << 32) + 300, 300
    p = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    g[-last:] = -0.25
    state = conv.adamw_state([p], bits)
    # (every step is lr whatever the gradient's size)
    conv.adamw([p], [g], state, 1, 0.5)
    conv.adamw([p], [g], state, 2, 0.25)
    assert bool((p[:-last] == 0.25).all()) and bool((p[-last:] == 1.75).all())
    del p, g, state
    torch.cuda.empty_cache()


# ---- refusals ---------------------------------------------------------------------------------

def test_python_refusals():
    x, w, wd = torch.zeros(70, 64, device=DEV), torch.zeros(40, 64, device=DEV), torch.zeros(64, 40, device=DEV)
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="ws"):
        conv.feed_forward_into(x, w, w, wd, y, None, None)
    with pytest.raises(ValueError, match="saved"):
        conv.feed_forward_into(x, w, w, wd, y, torch.empty(10, dtype=torch.uint8, device=DEV), None)
    with pytest.raises(ValueError, match="w_up"):
        conv.feed_forward(x, w, w.half(), wd)
    with pytest.raises(ValueError, match="dw_gate"):
        _, s = conv.feed_forward(x, w, w, wd)
        conv.feed_forward_backward_into(x, x, w, w, wd, s, y, w.half(), w, wd, None)
    for k, name in enumerate(("x", "w_gate", "w_up", "w_down")):
        big = [torch.zeros(t.shape[0], t.shape[1] + 8, device=DEV)[:, 1:1 + t.shape[1]] if i == k else t
               for i, t in enumerate((x, w, w, wd))]
        with pytest.raises(ValueError, match=f"^{name} must start on a 16-byte boundary"):
            conv.feed_forward(*big)
    with pytest.raises(ValueError, match="overlap|stride|contiguous"):
        conv.feed_forward(torch.zeros(1, 64, device=DEV).expand(70, 64), w, w, wd)
    r = torch.zeros(6, 32, device=DEV)
    with pytest.raises(ValueError, match="out must be"):
        conv.residual_norm_into(r, r, r.half(), r, None)
    with pytest.raises(ValueError, match="y must be"):
        conv.residual_norm_into(r, r, r.clone(), r[:3], None)
    with pytest.raises(ValueError, match="stats"):
        conv.residual_norm_into(r, r, r.clone(), r.clone(), torch.empty(6, 3, device=DEV))
    with pytest.raises(conv.Conv2dError, match="UNSUPPORTED"):
        conv.residual_norm(r, r.half())
    with pytest.raises(ValueError, match="weight"):
        conv.residual_norm(r, r, weight=torch.ones(31, device=DEV))
    with pytest.raises(ValueError, match="ws"):
        o, yy, st = conv.residual_norm(r, r)
        conv.residual_norm_backward_into(r, None, r, o, st, o.clone(), yy, None, dweight=torch.ones(32, device=DEV))
    state = conv.adamw_state([r])
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        conv.adamw([r], [r.t()], state, 1, 0.1)
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        conv.adamw([r], [r[:3]], state, 1, 0.1)
    with pytest.raises(TypeError, match="dtype"):
        conv.adamw([r], [r.double()], state, 1, 0.1)
    with pytest.raises(ValueError, match="step"):
        conv.adamw([r], [r], state, torch.ones(1, device=DEV), 0.1)
    with pytest.raises(conv.Conv2dError, match="INVALID"):
        conv.adamw([r], [r], state, 1, 0.1, beta1=1.0)


# ---- together: streams, graphs, repeatability, the example -------------------------------------

def _block_step(p, x, dy, state, step, dt, bits):
    """One training step of a residual block: norm, feed-forward, joint, gradients, AdamW."""
    f = {k: v.to(TYPES[dt]) for k, v in p.items() if k.startswith("w_")}
    h, mean, rstd = conv.layer_norm(x, p["gamma"], p["beta"], out_dtype=TYPES[dt])
    y, saved = conv.feed_forward(h, f["w_gate"], f["w_up"], f["w_down"])
    kw = dict(gate=p["gate"], post_weight=p["post"], weight=p["next"], kind="rms")
    out, z, st = conv.residual_norm(y, x, **kw)
    dr, db, g = conv.residual_norm_backward(dy, None, y, out, st, **kw)
    dh, dg, du, dd = conv.feed_forward_backward(db, h, f["w_gate"], f["w_up"], f["w_down"], saved)
    dx, dgamma, dbeta = conv.layer_norm_backward(dh, x, p["gamma"], mean, rstd)
    names = ["gamma", "beta", "w_gate", "w_up", "w_down", "gate", "post", "next"]
    grads = [dgamma, dbeta, dg, du, dd, g["gate"], g["post_weight"], g["weight"]]
    conv.adamw([p[n] for n in names], grads, state, step, 1e-2, weight_decay=0.01, seed=9)
    return [out, z, dr, db, dx] + grads


def _block_inputs(dt, bits, N=200, C=96, F=200):
    g = torch.Generator(device=DEV).manual_seed(4)

    def rnd(*s):
        return torch.randn(s, generator=g, device=DEV)
    p = {"gamma": torch.ones(C, device=DEV), "beta": torch.zeros(C, device=DEV), "gate": 0.5 + 0.1 * rnd(4, C),
         "post": torch.ones(C, device=DEV), "next": torch.ones(C, device=DEV), "w_gate": rnd(F, C) / C ** 0.5,
         "w_up": rnd(F, C) / C ** 0.5, "w_down": rnd(C, F) / F ** 0.5}
    names = ["gamma", "beta", "w_gate", "w_up", "w_down", "gate", "post", "next"]
    return p, rnd(N, C), rnd(N, C).to(TYPES[dt]), conv.adamw_state([p[n] for n in names], bits)


def _all_of(p, state):
    more = [state.exp_avg_scale, state.exp_avg_sq_scale] if state.bits == 8 else []
    return [t.clone() for t in list(p.values()) + [state.exp_avg, state.exp_avg_sq] + more]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_block_step_same_bits_on_any_stream(dt, bits):
    runs = []
    for k in range(3):
        p, x, dy, state = _block_inputs(dt, bits)
        s = torch.cuda.Stream() if k == 2 else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs = [o for t in (1, 2, 3) for o in _block_step(p, x, dy, state, t, dt, bits)]
            runs.append([o.clone() for o in outs] + _all_of(p, state))
        s.synchronize()
    assert all(bool(torch.isfinite(t.float()).all()) for t in runs[0])
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(other, runs[0]))


@pytest.mark.parametrize("bits", [32, 8])
def test_block_step_captured_and_replayed(bits):
    """The step's number, counted on the device, makes every replay the next step."""
    dt = "bf16"
    p, x, dy, state = _block_inputs(dt, bits)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    warm = _block_inputs(dt, bits)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _block_step(*warm, step + 1, dt, bits)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        out = _block_step(p, x, dy, state, step, dt, bits)
    q, x2, dy2, other = _block_inputs(dt, bits)
    for t in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        want = _block_step(q, x2, dy2, other, torch.tensor([t], device=DEV), dt, bits)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), f"replay {t}"
        assert all(torch.equal(a, b) for a, b in zip(_all_of(p, state), _all_of(q, other))), f"replay {t}"


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_example_block_head(dt):
    """The example's blocks run, and its gradients are those of the formulas: a directional
    difference of its loss in fp32, finite losses in every type."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block_head.py")
    spec = importlib.util.spec_from_file_location("train_block_head", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=5, dtype=TYPES[dt], classes=50, channels=64, hidden=96, blocks=2)
    assert len(losses) == 5 and all(np.isfinite(losses))
    if dt != "f32":
        return
    gen = torch.Generator(device=DEV).manual_seed(0)
    head = mod.BlockHead(channels=64, hidden=96, classes=50, blocks=2, dtype=torch.float32, device=DEV)
    x, labels = torch.randn(120, 64, generator=gen, device=DEV), torch.randint(-1, 50, (120,), generator=gen, device=DEV)
    _, grads = head.gradients(x, labels)
    e = [torch.randn(t.shape, generator=gen, device=DEV) * t.float().norm() / t.numel() ** 0.5 for t in head.params]
    start = [t.clone() for t in head.params]

    def f(h):
        for t, s0, d in zip(head.params, start, e):
            t.copy_(s0 + h * d)
        return head.gradients(x, labels)[0].double().item()
    want = sum((a.double() * d.double()).sum().item() for a, d in zip(grads, e))
    h = 2.0 ** -7
    # fourth-order differences of a loss of about 4 with error 2^-21 over 2h
    got = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
    assert abs(got - want) <= 2e-3 * max(1.0, abs(want)), (got, want)
