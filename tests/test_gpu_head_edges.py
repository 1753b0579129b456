"""Training-head kernels where they are easiest to get wrong: NaN logits, what
masked rows hold, logits of 10^9, roundings that have to cancel, very many
rows, and launches wider than one grid. Bounds as in test_gpu_head.py: u = 2^-24
is the unit roundoff of fp32, uo that of the stored type."""
import numpy as np
import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _lib
from oracle import head as ref
from test_gpu_head import DEV, SUB, TYPES, U, UO, _check_xent, _close, _say, _xent_case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.lib()


def _ulp_half(v, dt):
    """Half the spacing of the type's numbers at v (float64 in, float64 out)."""
    e = torch.frexp(v.abs())[1].double()               # |v| in [2^(e-1), 2^e)
    return torch.clamp(torch.exp2(e - 1) * UO[dt], min=SUB[dt])


@pytest.mark.parametrize("N", [1, 16, 40, 300])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_nan_weights_reach_every_loss(N, dt):
    """NaN in the weights of one class, or of all classes of a tile: every unmasked
    row's lse and loss are NaN, wherever its target lies; masked rows stay 0.
    257 classes leave the last one alone in a tile of 32, 64, 128 or 256."""
    for V, lo, hi in ((257, 256, 257), (600, 0, 256), (600, 256, 512), (1025, 1024, 1025), (70, 69, 70)):
        _say(f"NaN weights N={N} V={V} classes {lo}..{hi} {dt}")
        x, w, _, _ = _xent_case(N, V, 72, dt, seed=N + V)
        w[lo:hi, 5] = NAN
        t = torch.full((N,), 0 if lo else V - 1, dtype=torch.int64)
        if N > 3:
            t[3] = -1
        loss, lse = (v.cpu() for v in conv.linear_cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV)))
        ok = t >= 0
        assert bool(torch.isnan(lse[ok]).all()), "lse"
        assert bool(torch.isnan(loss[ok]).all()), "loss"
        assert not loss[~ok].any() and not lse[~ok].any()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_nan_features_reach_loss_and_lse_of_their_row_alone(dt):
    for N, V in ((1, 300), (9, 257), (40, 100), (300, 2000)):
        x, w, t, _ = _xent_case(N, V, 64, dt, seed=6)
        k = N // 2
        t[k] = 3
        x[k, 5] = NAN
        loss, lse = (v.cpu() for v in conv.linear_cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV)))
        for v in (loss, lse):
            bad = torch.isnan(v)
            assert bad[k] and int(bad.sum()) == 1, (N, V, int(bad.sum()))


# ---- what a gradient of one row does to the others -------------------------------------------


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("value", [INF, -INF, 1e30, NAN])
@pytest.mark.parametrize("N", [70, 40000])
def test_gradients_of_masked_rows_change_nothing(dt, value, N):
    x, w, t, up = _xent_case(N, 20, 24, dt, seed=3)
    up *= 1e-6                                          # small against the type: the common scale counts
    t[10], t[N - 1] = -1, 20
    args = [v.to(DEV) for v in (x, w, t)]
    _, lse = conv.linear_cross_entropy(*args)
    got = []
    for g in (0.0, value):
        up[10] = up[N - 1] = g
        got.append(conv.linear_cross_entropy_backward(up.to(DEV), *args, lse))
    for a, b, name in zip(*got, ("dx", "dw")):
        assert torch.equal(a, b), name
    assert bool(got[0][1].any())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_an_infinite_gradient_stays_in_its_row(dt):
    x, w, t, up = _xent_case(70, 20, 24, dt, seed=3)
    up *= 1e-6
    t[10] = 4
    args = [v.to(DEV) for v in (x, w, t)]
    _, lse = conv.linear_cross_entropy(*args)
    rest = torch.arange(70) != 10
    got = []
    for g in (0.0, INF):
        up[10] = g
        got.append(conv.linear_cross_entropy_backward(up.to(DEV), *args, lse)[0].cpu())
    assert torch.equal(got[0][rest], got[1][rest]) and bool(got[0][rest].any())
    assert not bool(torch.isfinite(got[1][10]).all())


# ---- logits far beyond fp32's integers ------------------------------------------------------


@pytest.mark.parametrize("N", [3, 40, 600])
@pytest.mark.parametrize("dt,exps", [("f32", (15, 20, 26, 31, 34, 60, 100)), ("bf16", (15, 20, 26, 31, 34, 60, 100)),
                                     ("f16", (15, 20, 26, 34))])
def test_equal_logits_of_any_size(N, dt, exps):
    """All logits equal 77/64 * 2^e exactly: the loss is log V for every e. From 2^31 on
    lse rounds to the logit itself, so that exp(l - lse) = 1 and the gradients are
    small integers times powers of two."""
    V, D = 100, 64
    for e in exps:
        _say(f"equal logits 2^{e} N={N} {dt}")
        a, b = 2.0 ** ((e - 6) // 2), 77 / 64 * 2.0 ** (e - 6 - (e - 6) // 2)
        x = torch.full((N, D), a).to(TYPES[dt]).to(DEV)
        w = torch.full((V, D), b).to(TYPES[dt]).to(DEV)
        t = torch.zeros(N, dtype=torch.int64, device=DEV)
        loss, lse = conv.linear_cross_entropy(x, w, t)
        # V exponentials of 0 in a chain of at most V / 64 + 64, logarithm and subtraction
        _close(loss, torch.full((N,), np.log(V), dtype=torch.float64), torch.tensor((V / 64 + 64 + 44) * U), "loss")
        want = 77 / 64 * 2.0 ** e + np.log(V)
        assert ((lse.cpu().double() - want).abs() <= 2 * U * want + 2e-5).all()
        if e < 31:
            continue
        assert bool((lse == 77 / 64 * 2.0 ** e).all())
        up = torch.full((N,), 2.0 ** -10, device=DEV)
        dx, dw = conv.linear_cross_entropy_backward(up, x, w, t, lse)
        dx0 = torch.full((N, D), 99 * 2.0 ** -10 * b, dtype=torch.float64)
        _close(dx, dx0, _ulp_half(dx0, dt) + 2 * V * U * dx0, "dx")
        dw0 = torch.full((V, D), N * 2.0 ** -10 * a, dtype=torch.float64)
        dw0[0] = 0
        _close(dw, dw0, _ulp_half(dw0, dt) + 2 * N * U * dw0, "dw")


# ---- wider than a launch ----------------------------------------------------------------------


def test_more_feature_maps_than_workgroups_of_a_launch():
    """2^24 + 5 maps of 2 x 2 positions are as many tiles of 256 threads: more
    than the 2^32 threads of a launch."""
    N, C = (1 << 24) + 5, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(N, C, 4, generator=g, device=DEV).half()
    w, b = torch.tensor([1.5, -0.5], device=DEV), torch.tensor([0.25, 1.0], device=DEV)
    kw = dict(layout="nchw", dropout_p=0.25, seed=3)
    y, mean, rstd = conv.layer_norm(x, w, b, **kw)
    # element 8 i begins map i: a half's own blocks begin at its first map
    for lo, hi in ((0, N // 2), (N // 2, N)):
        yh, mh, rh = conv.layer_norm(x[lo:hi], w, b, offset=lo, **kw)
        assert torch.equal(y[lo:hi], yh) and torch.equal(mean[lo:hi], mh) and torch.equal(rstd[lo:hi], rh)


def test_weight_gradient_of_no_rows_beyond_a_launch():
    V, D = (1 << 16) + 1, 1 << 16
    w = torch.empty(V, D, dtype=torch.bfloat16, device=DEV)
    dw = torch.ones_like(w)
    x = torch.empty(0, D, dtype=torch.bfloat16, device=DEV)
    z, e = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    conv.linear_cross_entropy_backward_into(e, x, w, z, e, torch.empty_like(x), dw, None)
    assert not bool(dw.any())


@pytest.mark.parametrize("layout,C", [("nhwc", (1 << 25) + 8), ("nchw", (1 << 26) + 4)])
def test_weight_gradients_of_more_channels_than_a_launch(layout, C):
    """One position of very many channels: the reductions of dweight and dbias."""
    g = torch.Generator(device=DEV).manual_seed(2)
    shape = (1, C) if layout == "nhwc" else (1, C, 1)
    x = torch.randn(shape, generator=g, device=DEV).half()
    dy = torch.randn(shape, generator=g, device=DEV).half()
    mean, rstd = torch.full((1,), 0.5, device=DEV), torch.full((1,), 2.0, device=DEV)
    if layout == "nchw":
        mean, rstd = mean.view(1, 1), rstd.view(1, 1)
    _, dw, db = conv.layer_norm_backward(dy, x, None, mean, rstd, layout=layout)
    want = dy.float().reshape(-1) * ((x.float().reshape(-1) - 0.5) * 2.0)
    # two products and a subtraction, rounded once each
    assert bool(((dw - want).abs() <= 4 * U * (want.abs() + dy.float().reshape(-1).abs())).all())
    assert torch.equal(db, dy.float().reshape(-1))


def test_more_logit_tiles_than_workgroups_of_a_launch():
    """2^22 rows by 65536 classes: 2^24 tiles of 128 x 128 with 256 threads, which is a
    grid of 2^32. Rows across the whole range against the definition."""
    N, V, D = 1 << 22, 65536, 320
    g = torch.Generator(device=DEV).manual_seed(3)
    w = (torch.randn(V, D, generator=g, device=DEV) * 0.1).bfloat16()
    x = torch.randn(N, D, generator=g, device=DEV, dtype=torch.bfloat16)
    t = torch.randint(0, V, (N,), generator=g, device=DEV)
    loss, lse = conv.linear_cross_entropy(x, w, t)
    assert bool(torch.isfinite(loss).all()) and bool((lse > 0).all())
    rows = torch.cat([torch.arange(500, device=DEV), torch.randint(0, N, (1000,), generator=g, device=DEV),
                      torch.arange(N - 500, N, device=DEV)])
    xs, ts = x[rows], t[rows]
    l0, s0 = ref.cross_entropy(xs, w, ts)
    dl = 2 * (D + 1) * U * (xs.double().abs() @ w.double().abs().t()).amax(1)
    tol = 2 * dl + (V / 64 + 108) * U + 4 * U * (2 * s0.abs() + l0.abs())
    _close(loss[rows], l0, tol, "loss")
    _close(lse[rows], s0, tol, "lse")


def test_views_that_start_off_a_granule_are_refused_by_name():
    """Rows of whole 16-byte granules are read in place and have to start on one."""
    x = torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    w = torch.zeros(5, 64, dtype=torch.float16, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    for a, b, name in ((x[:, 4:36], w[:, :32], "x"), (x[:, :32], w[:, 4:36], "w")):
        with pytest.raises(ValueError, match=f"^{name} must start on a 16-byte boundary"):
            conv.linear_cross_entropy(a, b, t)
    loss, lse = conv.linear_cross_entropy(x[:, :32], w[:, :32], t)
    with pytest.raises(ValueError, match="^w must start on a 16-byte boundary"):
        conv.linear_cross_entropy_backward(loss, x[:, :32], w[:, 4:36], t, lse)
    conv.linear_cross_entropy_backward(loss, x[:, 4:36], w[:, :32], t, lse)
    # rows that are copied first start anywhere
    conv.linear_cross_entropy(x[:, 3:34], w[:, 1:32], t)


def test_nchw_maps_without_positions():
    w = torch.ones(16, device=DEV)
    for shape in ((2, 16, 0), (2, 16, 0, 7)):
        x = torch.empty(shape, device=DEV)
        y, mean, rstd = conv.layer_norm(x, w, layout="nchw")
        assert y.shape == shape and mean.numel() == 0
        dx, dw, db = conv.layer_norm_backward(x, x, w, mean, rstd, layout="nchw")
        assert dx.shape == shape and not dw.any() and not db.any()


# ---- roundings of the gradient of the logits ---------------------------------------------------


@pytest.mark.parametrize("N,V,D", [(64, 30, 256), (300, 30, 100), (2100, 1700, 520), (16, 40000, 136), (5, 120, 1032),
                                   (700, 240, 72), (4100, 33000, 128), (40, 30, 101)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_an_offset_that_all_classes_share_cancels(N, V, D, dt):
    """sum_v G = 0 in every row, so a vector that all class weights share is not in
    dx. All logits are 0 here (x = 0) and every entry of G but the target's is 1/V,
    rounded the same way: unless G's roundings are made to cancel as G does, dx is
    off by that rounding times the offset. Bound: uo of G on the weights less
    their offset, the fp32 sums on the weights themselves, half a spacing of dx."""
    _say(f"shared offset N={N} V={V} D={D} {dt}")
    g = torch.Generator(device=DEV).manual_seed(N + V)
    off = torch.randn(1, D, generator=g, device=DEV)
    w = (torch.randn(V, D, generator=g, device=DEV) + 64.0 * off).to(TYPES[dt])
    x = torch.zeros(N, D, dtype=TYPES[dt], device=DEV)
    t = torch.randint(0, V, (N,), generator=g, device=DEV)
    up = torch.ones(N, device=DEV)
    _, lse = conv.linear_cross_entropy(x, w, t)
    dx, _ = conv.linear_cross_entropy_backward(up, x, w, t, lse)
    wd = w.double()
    mean = wd.mean(0, keepdim=True)
    dev = (wd - mean).abs()
    # G row by row: 1/V, and 1/V - 1 at the target; what the kernel takes as shared
    # lies within the spread of the class weights, feature by feature
    dx0 = mean - wd[t]
    uo = UO[dt] if dt != "f32" else 0.0
    rough = (dev.mean(0) + dev.amax(0)) * (uo * 1.01) + 2 * uo * uo * dev[t]
    # p's own error, (4 + |lse|) U of the type's fp32, times the offset; sums of V terms
    fine = (2 * (V / 64 + 64) + 48 + np.log(V)) * U * (wd.abs().mean(0) + wd.abs()[t]) if dt != "f32" else \
        (2 * (V + 8) + 48) * U * (wd.abs().mean(0) + wd.abs()[t])
    _close(dx, dx0, rough + fine + _ulp_half(dx0, dt), "dx")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_classes_apart_from_the_others_keep_their_bounds(dt):
    """Most class weights share an offset, but a row's few classes that count lie near 0
    in a feature: what the others share must not add to the error there. (With the
    least of 64 of the 150 classes taken as shared, the first of these exceeded it.)"""
    for seed in (113, 7, 50):
        x, w, t, up = _xent_case(100, 150, 3, dt, seed=983984738 + seed)
        g = torch.Generator().manual_seed(seed)
        w = (w.float() + 4 * torch.randn(1, 3, generator=g) * (2 / np.sqrt(3))).to(w.dtype)
        _check_xent(x, w, t, up, dt, ref_dev=DEV, what="classes apart", rel=False)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("N,V", [(512, 21), (512, 100), (600, 3000)])
def test_shared_offset_of_trained_weights(N, V, dt):
    """The same with rows that have logits: the relative L2 error of dx stays within
    that of rounding dx and G's entries on the centred weights."""
    D = 256
    g = torch.Generator(device=DEV).manual_seed(V)
    w = (torch.randn(V, D, generator=g, device=DEV) + 64.0 * torch.randn(1, D, generator=g, device=DEV)) / 8
    t = torch.randint(0, V, (N,), generator=g, device=DEV)
    x = torch.randn(N, D, generator=g, device=DEV) / 16
    x -= (x @ w.mean(0, keepdim=True).t()) @ w.mean(0, keepdim=True) / w.mean(0).norm() ** 2    # logits of order 1
    x, w = x.to(TYPES[dt]), w.to(TYPES[dt])
    up = torch.ones(N, device=DEV)
    _, lse = conv.linear_cross_entropy(x, w, t)
    dx, _ = conv.linear_cross_entropy_backward(up, x, w, t, lse)
    dx0, _, G = ref.cross_entropy_grad(up, x, w, t)
    far = G.abs()
    far[torch.arange(N, device=DEV), t] = 0
    wd = w.double()
    dev = (wd - wd.mean(0)).norm(dim=1)
    most = (wd - wd.mean(0)).abs().amax(0).norm()       # the mean against what is taken as shared
    logit = 2 * (D + 1) * U * (x.double().abs() @ wd.abs().t()).amax()         # p's relative error, all classes alike
    bound = UO[dt] * ((far @ dev + far.sum(1) * most) + dx0.norm(dim=1)) + \
        2 * logit * far.sum(1) * most + (2 * (V + 56) * U + 4 * U * (1 + lse.double().abs())) * (G.abs() @ wd.norm(dim=1))
    err = (dx.double() - dx0).norm(dim=1)
    _say(f"offset {N} {V} {dt}: relative L2 {((dx.double() - dx0).norm() / dx0.norm()).item():.2e}, "
         f"worst share of the bound {(err / bound).max().item():.2f}")
    assert bool((err <= bound).all())


@pytest.mark.parametrize("N,D,dt,V", [(64, 256, "bf16", 512), (300, 100, "bf16", 512), (2100, 520, "bf16", 512),
                                      (5000, 64, "bf16", 512), (64, 256, "f16", 4096), (2100, 136, "f16", 4096)])
def test_rounding_at_the_target_is_taken_back(N, D, dt, V):
    """With all logits 0, G is 1/V but at the target, where 1 - 1/V lies halfway
    between two numbers of the type. dx (from x = 0) and dw (from w = 0) have to be as
    good as with an unrounded G: half a spacing of the result, the fp32 sums'
    bounds, and the rounding of the target's remainder, uo / V of each row's
    contribution. The rounding itself, 1 / V, is a multiple of those."""
    _say(f"target rounding N={N} V={V} D={D} {dt}")
    g = torch.Generator(device=DEV).manual_seed(N)
    t = torch.randint(0, V, (N,), generator=g, device=DEV)
    up = torch.full((N,), 1.0, device=DEV)
    a = torch.randn(N, D, generator=g, device=DEV).to(TYPES[dt])
    b = torch.randn(V, D, generator=g, device=DEV).to(TYPES[dt])
    for x, w in ((torch.zeros_like(a), b), (a, torch.zeros_like(b))):
        _, lse = conv.linear_cross_entropy(x, w, t)
        dx, dw = conv.linear_cross_entropy_backward(up, x, w, t, lse)
        dx0, dw0, G = ref.cross_entropy_grad(up, x, w, t)
        far = G.abs()
        far[torch.arange(N, device=DEV), t] = 0         # exact in the type up to p's fp32 error
        X, W = x.double().abs(), w.double().abs()
        tol = _ulp_half(dx0, dt) + 2 * (V + 56) * U * (G.abs() @ W) + UO[dt] / V * W[t]
        _close(dx, dx0, tol, "dx")
        hit = torch.zeros(V, D, dtype=torch.float64, device=DEV).index_add_(0, t, X)
        tol = _ulp_half(dw0, dt) + 2 * (N + 56) * U * (G.abs().t() @ X) + UO[dt] / V * hit
        _close(dw, dw0, tol, "dw")


# ---- rows in numbers ------------------------------------------------------------------------


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,V,D", [(100352, 21, 256), (100352, 150, 256), (40001, 9, 24)])
def test_pixels_of_a_batch(N, V, D, dt):
    """As many rows as a batch has pixels, few classes; the largest row gradient
    comes late in the array."""
    x, w, t, up = _xent_case(N, V, D, dt, seed=V)
    up[N - 2] *= 50.0
    t[N - 2] = 1
    _check_xent(x, w, t, up, dt, ref_dev=DEV, what="pixels")


def test_row_weights_of_a_millionth_in_fp16():
    """Scaled into fp16's range, G keeps its digits; dx and dw below 2^-14 lose theirs
    in their own storage alone."""
    x, w, t, up = _xent_case(64, 1000, 128, "f16", seed=10)
    _check_xent(x, w, t, up * 1e-6, "f16", what="row weights of 1e-6", rel=False)
