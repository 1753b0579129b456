"""Training-head kernels (layer norm, dropout, linear cross entropy) against
their plain 64-bit forms (oracle/head.py), element by element.

Tolerances, derived from the operations (u = 2^-24, the unit roundoff of fp32;
uo that of the output's type, sub half its smallest subnormal): a sum of terms
added along chains of at most n fp32 additions is within n*u*sum|terms| of the
exact one (Higham, "Accuracy and Stability of Numerical Algorithms", ch. 4), and
every other operation adds a few u of its result. Chains: over the channels
of one position at most C/32 + 64, over positions at most N*P/64 + 256, over
the K of a matrix product at most K (times 2 for matrix cores that truncate),
over the classes of a row at most V/64 + 64. exp of an argument a is within
(4 + |a|) u."""
import numpy as np
import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _lib
from oracle import head as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UO = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
REL = {"f32": 1e-5, "f16": 2e-3, "bf16": 1e-2}     # relative L2 error, as for the convolution
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.lib()


def _say(msg):
    print(msg, flush=True)


def _close(got, want, tol, what):
    got, want = got.detach().cpu().double(), want.cpu().double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} against {tuple(want.shape)}"
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    err = (got - want).abs()
    bad = err > tol.cpu()
    if bad.any():
        i = torch.nonzero(bad.reshape(-1))[0].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; at {i}: got "
                             f"{got.reshape(-1)[i].item()!r}, exact {want.reshape(-1)[i].item()!r}, bound "
                             f"{tol.expand_as(err).reshape(-1)[i].item():.3e}")


def _rel(got, want, dt, what):
    got, want = got.detach().cpu().double(), want.cpu().double()
    den = want.norm()
    if den > 0:
        rel = ((got - want).norm() / den).item()
        assert rel <= REL[dt], f"{what}: relative L2 error {rel:.3e}"


# ---- layer norm --------------------------------------------------------------------

def _vec(v, dim, nd):
    return v.double().reshape([-1 if i == dim else 1 for i in range(nd)])


def _norm_case(shape, dim, xt, yt, seed, affine=True):
    g = torch.Generator().manual_seed(seed)
    C = shape[dim]
    lev = torch.randn([C if i == dim else 1 for i in range(len(shape))], generator=g)
    x = (torch.randn(shape, generator=g) * 1.5 + 2.0 * lev).to(TYPES[xt])
    dy = torch.randn(shape, generator=g).to(TYPES[yt])
    w = 1.0 + 0.3 * torch.randn(C, generator=g) if affine else None
    b = 0.5 * torch.randn(C, generator=g) if affine else None
    return x, dy, w, b


def _check_norm(shape, layout, xt, yt, p=0.0, seed=3, affine=True, eps=1e-5):
    nchw = layout == "nchw"
    dim = 1 if nchw else len(shape) - 1
    nd = len(shape)
    x, dy, w, b = _norm_case(shape, dim, xt, yt, seed, affine)
    C = shape[dim]
    pos = int(np.prod(shape)) // C
    sd, off = 0xABCDEF0123456789 - seed, (1 << 33) + 5
    _say(f"layer norm {layout} {shape} {xt}->{yt} p={p} affine={affine}")
    xd, dyd = x.to(DEV), dy.to(DEV)
    wd, bd = (w.to(DEV), b.to(DEV)) if affine else (None, None)
    y, mean, rstd = conv.layer_norm(xd, wd, bd, eps, layout=layout, out_dtype=TYPES[yt], dropout_p=p, seed=sd,
                                    offset=off)
    torch.cuda.synchronize()
    y0, m0, r0 = ref.layer_norm(x, w, b, eps, dim)
    drop = ref.drop_factors(shape, p, sd, off)
    X = x.double()
    D1, D2 = C / 32 + 64, pos / 64 + 256
    dm = D1 * U * X.abs().mean(dim) + U * m0.abs()
    _close(mean, m0, dm, "mean")
    rho = 0.5 * ((D1 + 4) * U + (dm * r0) ** 2) + 4 * U
    _close(rstd, r0, rho * r0, "rstd")
    W = _vec(w, dim, nd) if affine else torch.ones(1, dtype=torch.float64)
    B = _vec(b, dim, nd) if affine else torch.zeros(1, dtype=torch.float64)
    r, dmu = r0.unsqueeze(dim), dm.unsqueeze(dim)
    h = (X - m0.unsqueeze(dim)) * r
    tol = W.abs() * r * dmu + (h * W).abs() * (rho.unsqueeze(dim) + 6 * U) + 4 * U * (y0.abs() + B.abs())
    want = y0 * drop
    _close(y, want, tol * drop + UO[yt] * want.abs() * 1.01 + SUB[yt], "y")
    assert (y.cpu()[drop == 0] == 0).all()
    _rel(y, want, yt, "y")

    dx, dw, db = conv.layer_norm_backward(dyd, xd, wd, mean, rstd, layout=layout, dropout_p=p, seed=sd, offset=off)
    torch.cuda.synchronize()
    mc, rc = mean.cpu(), rstd.cpu()
    dz = dy.double() * drop
    dx0, dw0, db0 = ref.layer_norm_grad(dz, x, w, mc, rc, dim)
    r = rc.double().unsqueeze(dim)
    h = (X - mc.double().unsqueeze(dim)) * r
    gabs = (dz * W).abs()
    e1 = (D1 + 5) * U * gabs.mean(dim, keepdim=True)
    e2 = (D1 + 9) * U * (gabs * h.abs()).mean(dim, keepdim=True)
    s2 = (dz * W * h).mean(dim, keepdim=True).abs()
    s1 = (dz * W).mean(dim, keepdim=True).abs()
    tol = r * (e1 + h.abs() * e2 + 10 * U * (gabs + s1 + h.abs() * s2)) + UO[xt] * dx0.abs() * 1.01 + SUB[xt]
    _close(dx, dx0, tol, "dx")
    rest = [i for i in range(nd) if i != dim]

    def tot(t):
        return t.sum(rest) if rest else t
    _close(dw, dw0, (D2 + 8) * U * tot((dz * h).abs()), "dweight")
    _close(db, db0, (D2 + 4) * U * tot(dz.abs()), "dbias")
    _rel(dx, dx0, xt, "dx")


COMBOS = [("f32", "f32"), ("f32", "f16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "bf16")]


@pytest.mark.parametrize("N,C", [(1, 1), (3, 7), (1, 8), (70, 64), (33, 65), (9, 120), (50, 128), (7, 250),
                                 (65, 256), (5, 511), (130, 512), (3, 1000), (17, 1024), (4, 1025), (600, 2048),
                                 (5, 2056), (6, 4096), (3, 5001), (2, 8192), (3, 8200), (2, 20011)])
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16")], ids="-".join)
def test_layer_norm_rows(N, C, types):
    _check_norm((N, C), "nhwc", *types, seed=N + C)


@pytest.mark.parametrize("types", COMBOS, ids="-".join)
@pytest.mark.parametrize("C,p", [(64, 0.1), (77, 0.5), (1032, 0.1), (4001, 0.25), (9000, 0.1), (9001, 0.3)])
def test_layer_norm_rows_types_and_dropout(C, types, p):
    _check_norm((2, 3, 4, C), "nhwc", *types, p=p, seed=C)


@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 3, 7, 7), (3, 32, 64), (2, 64, 14, 14), (5, 65, 49), (1, 130, 13, 5),
                                   (2, 256, 7, 7), (2, 500, 31), (1, 512, 196), (2, 513, 50), (3, 700, 9),
                                   (40, 64, 28, 28)])
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16")], ids="-".join)
def test_layer_norm_nchw(shape, types):
    _check_norm(shape, "nchw", *types, seed=sum(shape))


@pytest.mark.parametrize("types", COMBOS, ids="-".join)
@pytest.mark.parametrize("shape,p", [((2, 33, 7, 7), 0.5), ((2, 64, 14, 14), 0.1), ((2, 100, 12), 0.1),
                                     ((1, 520, 26), 0.25), ((3, 600, 7, 7), 0.1), ((4, 96, 56, 8), 0.2)])
def test_layer_norm_nchw_types_and_dropout(shape, types, p):
    _check_norm(shape, "nchw", *types, p=p, seed=sum(shape))


def test_layer_norm_without_weight_and_stats():
    _check_norm((9, 100), "nhwc", "f16", "f16", affine=False)
    _check_norm((2, 40, 9), "nchw", "f32", "f32", affine=False)
    _check_norm((2, 9001), "nhwc", "bf16", "bf16", affine=False)
    x = torch.randn(5, 64, device=DEV)
    y = torch.empty_like(x)
    conv.layer_norm_into(x, None, None, y, None, None)
    assert torch.equal(y, conv.layer_norm(x)[0])


def test_layer_norm_constant_rows_and_large_offsets():
    """A constant row gives y = bias; a level far above the spread keeps the
    two-pass variance."""
    x = torch.full((4, 96), 3.0, device=DEV)
    b = torch.randn(96, device=DEV)
    y, mean, rstd = conv.layer_norm(x, None, b)
    assert torch.equal(y, b.expand(4, 96)) and bool((mean == 3.0).all())
    assert torch.allclose(rstd, torch.full((4,), 1e-5, device=DEV).rsqrt(), rtol=1e-6)
    g = torch.Generator().manual_seed(5)
    x = 1000.0 + torch.randn(6, 640, generator=g)
    y, _, _ = conv.layer_norm(x.to(DEV))
    y0, m0, r0 = ref.layer_norm(x, None, None, 1e-5, 1)
    # the mean is off by at most (C/32 + 64) u * 1000, divided by a deviation of 1
    _close(y, y0, (84 * U * 1001.0 * 1.2) * torch.ones_like(y0) + 1e-5 * y0.abs(), "y")


def test_layer_norm_strided_rows_leave_the_gaps():
    g = torch.Generator().manual_seed(11)
    for C, ld, off, dt in ((100, 131, 3, torch.float16), (64, 72, 8, torch.bfloat16), (300, 301, 1, torch.float32)):
        big = torch.randn(10, ld, generator=g).to(dt).to(DEV)
        x = big[:, off:off + C] if off + C <= ld else big[:, :C]
        w = torch.randn(C, generator=g).to(DEV)
        ybig = torch.full((10, ld + 5), 7.0, dtype=dt, device=DEV)
        y = ybig[:, 2:2 + C]
        mean, rstd = torch.empty(10, device=DEV), torch.empty(10, device=DEV)
        conv.layer_norm_into(x, w, None, y, mean, rstd, dropout_p=0.25, seed=4)
        xc = x.contiguous()
        y1, m1, r1 = conv.layer_norm(xc, w, dropout_p=0.25, seed=4)
        assert torch.equal(y, y1) and torch.equal(mean, m1) and torch.equal(rstd, r1)
        assert bool((ybig[:, :2] == 7).all()) and bool((ybig[:, 2 + C:] == 7).all())
        dxbig = torch.full((10, ld + 3), 5.0, dtype=dt, device=DEV)
        dx = dxbig[:, 1:1 + C]
        dw, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        ws = torch.empty(conv.layer_norm_workspace_size(x), dtype=torch.uint8, device=DEV)
        conv.layer_norm_backward_into(y, x, w, mean, rstd, dx, dw, db, ws, dropout_p=0.25, seed=4)
        a, b, c = conv.layer_norm_backward(y1, xc, w, m1, r1, dropout_p=0.25, seed=4)
        assert torch.equal(dx, a) and torch.equal(dw, b) and torch.equal(db, c)
        assert bool((dxbig[:, 0] == 5).all()) and bool((dxbig[:, 1 + C:] == 5).all())
    # leading dimensions collapse into rows of one stride, or are refused
    t = torch.randn(3, 4, 20, device=DEV)[:, :, :12]
    assert torch.equal(conv.layer_norm(t)[0], conv.layer_norm(t.contiguous())[0])
    with pytest.raises(ValueError, match="one stride"):
        conv.layer_norm(torch.randn(3, 5, 20, device=DEV)[:, :4])


def test_layer_norm_nan_stays_in_its_position():
    x = torch.randn(8, 200, device=DEV)
    x[3, 17] = float("nan")
    y, _, _ = conv.layer_norm(x)
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isfinite(y[[0, 1, 2, 4, 5, 6, 7]]).all())
    x = torch.randn(2, 40, 30, device=DEV)
    x[1, 5, 7] = float("inf")
    y, _, _ = conv.layer_norm(x, layout="nchw")
    bad = ~torch.isfinite(y)
    assert bool(bad[1, :, 7].all()) and int(bad.sum()) == 40


def test_layer_norm_empty():
    w = torch.ones(16, device=DEV)
    x = torch.empty(0, 16, device=DEV)
    y, mean, rstd = conv.layer_norm(x, w)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = conv.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    x = torch.empty(0, 16, 5, device=DEV)
    y, mean, rstd = conv.layer_norm(x, w, layout="nchw")
    dx, dw, db = conv.layer_norm_backward(x, x, w, mean, rstd, layout="nchw")
    assert not dw.any() and not db.any()
    for C in (9001,):
        x = torch.empty(0, C, device=DEV)
        e = torch.empty(0, device=DEV)
        _, dw, db = conv.layer_norm_backward(x, x, None, e, e)
        assert not dw.any() and not db.any()


# ---- dropout -------------------------------------------------------------------------

@pytest.mark.parametrize("n", [0, 1, 7, 8, 9, 1000, 4097, 300001])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_dropout_is_the_definition_bit_for_bit(n, dt):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(TYPES[dt])
    for p, seed, off in ((0.1, 5, 0), (0.5, (1 << 64) - 3, (1 << 64) - 4), (0.0, 1, 1), (1.0, 1, 1)):
        _say(f"dropout {dt} n={n} p={p}")
        y = conv.dropout(x.to(DEV), p, seed, off).cpu()
        f = ref.drop_factors((n,), p, seed, off) if n else torch.empty(0, dtype=torch.float64)
        want = torch.where(f > 0, x.float() * f.float(), torch.zeros(())).to(TYPES[dt])
        assert torch.equal(y, want)


def test_dropout_drops_nan_and_infinities_and_works_in_place_and_unaligned():
    x = torch.full((4096,), float("nan"), device=DEV)
    x[::2] = float("inf")
    f = ref.drop_factors((4096,), 0.5, 77, 3).to(DEV)
    y = conv.dropout(x, 0.5, 77, 3)
    assert bool((y[f == 0] == 0).all()) and not bool(torch.isfinite(y[f > 0]).any())
    z = torch.randn(5001, device=DEV).half()
    want = conv.dropout(z[1:].contiguous(), 0.25, 9)
    a = z.clone()
    conv.dropout_into(a[1:], a[1:], 0.25, 9)
    assert torch.equal(a[1:], want) and a[0] == z[0]


def test_dropout_gradient_is_the_same_map():
    """dropout is linear with a fixed mask: <dropout(x), dy> = <x, dropout(dy)>."""
    g = torch.Generator(device=DEV).manual_seed(4)
    x, dy = (torch.randn(10007, generator=g, device=DEV) for _ in range(2))
    a = (conv.dropout(x, 0.3, 8).double() * dy.double()).sum().item()
    b = (x.double() * conv.dropout(dy, 0.3, 8).double()).sum().item()
    # each product is rounded once in fp32 on either side
    assert abs(a - b) <= 2 * U * (x.double() * dy.double()).abs().sum().item() / 0.7


def test_fused_dropout_equals_dropout_of_the_norm():
    x = torch.randn(50, 77, device=DEV)
    y = conv.layer_norm(x)[0]
    assert torch.equal(conv.layer_norm(x, dropout_p=0.3, seed=5, offset=2)[0], conv.dropout(y, 0.3, 5, 2))
    x = torch.randn(3, 20, 11, device=DEV)
    y = conv.layer_norm(x, layout="nchw")[0]
    assert torch.equal(conv.layer_norm(x, layout="nchw", dropout_p=0.3, seed=5)[0], conv.dropout(y, 0.3, 5))


# channels on both sides of each number that a kernel holds, positions that are and
# are not whole tiles, vectors and 8-element blocks; the third has more tiles than
# workgroups
@pytest.mark.parametrize("N,C,P", [(3, 36, 49), (2, 64, 196), (601, 70, 26), (3, 129, 47), (2, 257, 64), (5, 512, 33),
                                   (3, 513, 49), (40, 700, 98), (2, 1024, 17), (2, 1025, 21), (7, 300, 3), (4, 90, 4)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_fused_dropout_of_feature_maps(N, C, P, dt):
    _say(f"layer norm nchw dropout {N} {C} {P} {dt}")
    g = torch.Generator(device=DEV).manual_seed(N + C + P)
    x = torch.randn(N, C, P, generator=g, device=DEV).to(TYPES[dt])
    dy = torch.randn(N, C, P, generator=g, device=DEV)
    w, b = torch.randn(C, generator=g, device=DEV), torch.randn(C, generator=g, device=DEV)
    y, mean, rstd = conv.layer_norm(x.float(), w, b, layout="nchw")
    kw = {"layout": "nchw", "dropout_p": 0.3, "seed": 11, "offset": 3}
    assert torch.equal(conv.layer_norm(x.float(), w, b, **kw)[0], conv.dropout(y, 0.3, 11, 3))
    got = conv.layer_norm_backward(dy, x.float(), w, mean, rstd, **kw)
    want = conv.layer_norm_backward(conv.dropout(dy, 0.3, 11, 3), x.float(), w, mean, rstd, layout="nchw")
    # the same fp32 formula twice: sums of up to 16016 terms in one order or another,
    # 16016 U < 2e-3 of the terms' magnitudes, in practice far less; a wrong mask is O(1)
    for a, c in zip(got, want):
        assert (a - c).abs().max().item() <= 1e-4 * c.abs().max().item()
    if dt == "bf16":
        yb = conv.layer_norm(x, w, b, layout="nchw")[0]
        yd = conv.layer_norm(x, w, b, **kw)[0]
        assert torch.equal(yd == 0, (conv.dropout(yb, 0.3, 11, 3) == 0))


# ---- linear cross entropy ----------------------------------------------------------------

def _xent_case(N, V, D, dt, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(V, D, generator=g) * (spread / np.sqrt(D))
    t = torch.randint(0, V, (N,), generator=g)
    x = (torch.randn(N, D, generator=g) + w[t] * 1.5).to(TYPES[dt])
    t[torch.rand(N, generator=g) < 0.1] = -1
    if N > 2:
        t[0], t[1], t[2] = 0, V - 1, V
    # unequal row weights; fp16 with the loss scale of half-precision training
    up = torch.rand(N, generator=g) + 0.5
    return x, w.to(TYPES[dt]), t, up if dt == "f16" else up / N


def _check_xent(x, w, t, up, dt, ref_dev="cpu", what="", rel=True):
    N, D = x.shape
    V = w.shape[0]
    _say(f"linear cross entropy {what} N={N} V={V} D={D} {dt}")
    xd, wd, td, ud = x.to(DEV), w.to(DEV), t.to(DEV), up.to(DEV)
    loss, lse = conv.linear_cross_entropy(xd, wd, td)
    dx, dw = conv.linear_cross_entropy_backward(ud, xd, wd, td, lse)
    torch.cuda.synchronize()
    x, w, t, up = (v.to(ref_dev) for v in (x, w, t, up))
    l0, s0 = ref.cross_entropy(x, w, t)
    ok = (t >= 0) & (t < V)
    X = torch.where(ok[:, None], x.double(), 0.0).abs()
    Wa = w.double().abs()
    dl = 2 * (D + 1) * U * (X @ Wa.t())                    # every logit
    di = dl.amax(1)
    esum = (V / 64 + 64 + 44) * U
    ts = torch.where(ok, di + esum + 2 * U * s0.abs(), 0.0)
    _close(lse, s0, ts, "lse")
    tl = torch.where(ok, 2 * di + esum + 4 * U * (s0.abs() + (s0 - l0).abs()), 0.0)
    _close(loss, l0, tl, "loss")
    lse_in = lse.to(ref_dev)
    dx0, dw0, G = ref.cross_entropy_grad(up, x, w, t, lse_in)
    p = torch.exp(torch.where(ok[:, None], x.double(), 0.0) @ w.double().t() - lse_in.double()[:, None])
    g = up.double().abs()[:, None] * ok[:, None]
    gmax = up.double().abs().max()
    # G below the normal range of the type it is held in: fp16's smallest
    # subnormal against the largest row weight, 2^-126 for the others
    low = gmax * 2.0 ** -39 if dt == "f16" else 2.0 ** -126
    dG = g * p * (dl + 48 * U) + 4 * U * G.abs() + (UO[dt] * G.abs() * 1.01 + low) * ok[:, None]
    tol = dG @ Wa + 2 * (V + 8) * U * (G.abs() @ Wa) + UO[dt] * dx0.abs() * 1.01 + SUB[dt]
    _close(dx, dx0, tol * ok[:, None], "dx")
    tol = dG.t() @ X + 2 * (N + 8) * U * (G.abs().t() @ X) + UO[dt] * dw0.abs() * 1.01 + SUB[dt]
    _close(dw, dw0, tol, "dw")
    if rel:
        _rel(loss, l0, "f32", "loss")
        _rel(dx, dx0, dt, "dx")
        _rel(dw, dw0, dt, "dw")


XENT = [(1, 1, 1), (1, 10, 7), (2, 300, 64), (3, 100, 64), (16, 257, 128), (17, 3001, 8), (64, 1000, 512),
        (65, 129, 72), (100, 2000, 250), (130, 257, 96), (257, 513, 260), (300, 70, 1032), (5, 20000, 64),
        (31, 4099, 321), (520, 1500, 576)]


@pytest.mark.parametrize("N,V,D", XENT)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_cross_entropy(N, V, D, dt):
    _check_xent(*_xent_case(N, V, D, dt, seed=N + V + D), dt)


@pytest.mark.parametrize("N,V,D,dt", [(4100, 33000, 128, "bf16"), (2050, 40001, 72, "f32"), (4100, 33000, 200, "f16")])
def test_linear_cross_entropy_in_several_pieces(N, V, D, dt):
    """Enough rows x classes that the backward pass takes more than one piece."""
    _check_xent(*_xent_case(N, V, D, dt, seed=1), dt, ref_dev=DEV, what="pieces")


@pytest.mark.parametrize("N,V,D", [(2100, 9000, 520), (3000, 40, 200), (2500, 130, 264), (16, 40000, 264),
                                   (700, 33000, 260), (1, 70001, 136), (200, 100, 4096), (33, 300, 2500)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_cross_entropy_tile_shapes(N, V, D, dt):
    """Many tiles per workgroup, targets in every block of G, few rows against
    many classes, long K split over workgroups and over waves."""
    _check_xent(*_xent_case(N, V, D, dt, seed=N), dt, ref_dev=DEV, what="tiles")


@pytest.mark.parametrize("N,V,D", [(1601, 208, 376), (2300, 384, 1000), (2300, 384, 2600), (4099, 5, 48), (129, 33, 2048)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_cross_entropy_with_few_classes(N, V, D, dt):
    """Every stage of rows then has a target among every wave's classes."""
    _check_xent(*_xent_case(N, V, D, dt, seed=9), dt, ref_dev=DEV, what="few classes")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_linear_cross_entropy_strided_and_unaligned(dt):
    N, V, D = 70, 300, 104
    x, w, t, up = _xent_case(N, V, D, dt, seed=9)
    want = None
    for lx, ox, lw, ow in ((D, 0, D, 0), (D + 8, 8, D + 24, 16), (D + 3, 1, D, 0), (D, 0, D + 5, 3), (D + 1, 1, D + 1, 0)):
        bx, bw = torch.full((N, lx), float("nan")).to(x.dtype), torch.full((V, lw), float("nan")).to(w.dtype)
        bx[:, ox:ox + D], bw[:, ow:ow + D] = x, w
        xs, wsl = bx.to(DEV)[:, ox:ox + D], bw.to(DEV)[:, ow:ow + D]
        loss, lse = conv.linear_cross_entropy(xs, wsl, t.to(DEV))
        dx, dw = conv.linear_cross_entropy_backward(up.to(DEV), xs, wsl, t.to(DEV), lse)
        got = [v.cpu() for v in (loss, lse, dx, dw)]
        if want is None:
            _check_xent(x, w, t, up, dt)
            want = got
        for a, b, name in zip(got, want, ("loss", "lse", "dx", "dw")):
            assert torch.equal(a, b), f"{name} differs for strides {lx}+{ox}, {lw}+{ow}"


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_masked_rows_may_hold_anything(dt):
    x, w, t, up = _xent_case(70, 200, 72, dt, seed=3)
    t[10:13] = torch.tensor([-100, 200, -(1 << 62)])
    up[11] = float("nan")
    clean = x.clone()
    clean[10:13] = 0
    x[10], x[11], x[12] = float("nan"), float("inf"), float("-inf")
    uc = torch.where(torch.isnan(up), torch.zeros(()), up)
    a = conv.linear_cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV))
    b = conv.linear_cross_entropy(clean.to(DEV), w.to(DEV), t.to(DEV))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ga = conv.linear_cross_entropy_backward(up.to(DEV), x.to(DEV), w.to(DEV), t.to(DEV), a[1])
    gb = conv.linear_cross_entropy_backward(uc.to(DEV), clean.to(DEV), w.to(DEV), t.to(DEV), a[1])
    for p, q in zip(ga, gb):
        assert torch.equal(p, q) and bool(torch.isfinite(p).all())
    assert not ga[0][10:13].any()


def test_all_rows_masked_and_no_rows():
    for dt in ("f32", "f16", "bf16"):
        x, w, t, up = _xent_case(20, 50, 24, dt, seed=3)
        t[:] = -1
        loss, lse = conv.linear_cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV))
        dx, dw = conv.linear_cross_entropy_backward(up.to(DEV), x.to(DEV), w.to(DEV), t.to(DEV), lse)
        assert not loss.any() and not lse.any() and not dx.any() and not dw.any()
        e = torch.empty(0, 24, dtype=TYPES[dt], device=DEV)
        z = torch.empty(0, dtype=torch.int64, device=DEV)
        loss, lse = conv.linear_cross_entropy(e, w.to(DEV), z)
        dx, dw = conv.linear_cross_entropy_backward(loss, e, w.to(DEV), z, lse)
        assert loss.shape == (0,) and dx.shape == (0, 24) and not dw.any()


def test_unmasked_nan_row_stays_in_its_row():
    x, w, t, up = _xent_case(40, 100, 64, "bf16", seed=6)
    t[7] = 3
    x[7, 5] = float("nan")
    loss, _ = conv.linear_cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV))
    bad = torch.isnan(loss).cpu()
    assert bad[7] and int(bad.sum()) == 1


@pytest.mark.parametrize("scale", [30.0, 3000.0])
def test_large_logits(scale):
    """Logits of thousands: the running maximum keeps the sums finite. The
    relative L2 figures do not apply: an fp32 logit of 1e5 is itself uncertain by
    1e-2, which the bounds of each element carry."""
    for dt in ("f32", "bf16"):
        x, w, t, up = _xent_case(33, 500, 64, dt, seed=8)
        _check_xent((x.float() * scale).to(x.dtype), w, t, up, dt, what=f"x {scale}", rel=False)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_small_losses_of_large_logits(dt):
    """Logits a for the target and a - 16 for 99 others, all exact: the loss,
    log(1 + 99 exp(-16)), is far below the spacing of fp32 numbers near a."""
    a = torch.tensor([1000.0, 992.0, 512.0, 64.0])
    x = torch.stack([a, a - 16], 1).to(TYPES[dt]).to(DEV)
    w = torch.zeros(100, 2)
    w[0, 0], w[1:, 1] = 1, 1
    loss, lse = conv.linear_cross_entropy(x, w.to(TYPES[dt]).to(DEV), torch.zeros(4, dtype=torch.int64, device=DEV))
    # a sum of exponentials near 1 by at most 40 additions, its logarithm, a subtraction
    want = float(np.log1p(99 * np.exp(-16.0)))
    assert (loss.cpu().double() - want).abs().max().item() <= 44 * U
    assert ((lse.cpu().double() - a.double() - want).abs() <= 2 * U * a.double()).all()


def test_zero_gradient_rows():
    x, w, t, up = _xent_case(33, 500, 64, "f16", seed=8)
    loss, lse = conv.linear_cross_entropy(x.to(DEV), w.to(DEV), t.to(DEV))
    dx, dw = conv.linear_cross_entropy_backward(torch.zeros(33, device=DEV), x.to(DEV), w.to(DEV), t.to(DEV), lse)
    assert not dx.any() and not dw.any()


def test_small_row_weights_in_fp16():
    """Row weights of 1e-6: the gradient's type underflows them only in dx and dw themselves."""
    x, w, t, up = _xent_case(64, 1000, 128, "f16", seed=10)
    _check_xent(x, w, t, up * 1e-2, "f16", what="small row weights")


def test_gradients_against_differences():
    """Directional differences of the fp32 loss through the kernels themselves."""
    x, w, t, up = _xent_case(40, 300, 96, "f32", seed=12)
    xd, wd, td, ud = x.to(DEV), w.to(DEV), t.to(DEV), up.to(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    ex = torch.randn(xd.shape, generator=g, device=DEV)
    ew = torch.randn(wd.shape, generator=g, device=DEV) * 0.1

    def f(h):
        return (conv.linear_cross_entropy(xd + h * ex, wd + h * ew, td)[0].double() * ud.double()).sum().item()
    _, lse = conv.linear_cross_entropy(xd, wd, td)
    dx, dw = conv.linear_cross_entropy_backward(ud, xd, wd, td, lse)
    want = ((dx.double() * ex.double()).sum() + (dw.double() * ew.double()).sum()).item()
    h = 2.0 ** -7
    # fourth-order differences: losses of about 7 with error 2^-20 over 2h, truncation h^4 times the fifth derivative
    got = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
    assert abs(got - want) <= 2e-3 * max(1.0, abs(want)), (got, want)

    xn = torch.randn(30, 100, generator=g, device=DEV)
    wt, b = torch.randn(100, generator=g, device=DEV), torch.randn(100, generator=g, device=DEV)
    dy, e = torch.randn(30, 100, generator=g, device=DEV), torch.randn(30, 100, generator=g, device=DEV)
    kw = dict(dropout_p=0.2, seed=3)

    def n(h):
        return (conv.layer_norm(xn + h * e, wt, b, **kw)[0].double() * dy.double()).sum().item()
    _, mean, rstd = conv.layer_norm(xn, wt, b, **kw)
    dxn, _, _ = conv.layer_norm_backward(dy, xn, wt, mean, rstd, **kw)
    want = (dxn.double() * e.double()).sum().item()
    got = (8 * (n(h) - n(-h)) - (n(2 * h) - n(-2 * h))) / (12 * h)
    assert abs(got - want) <= 2e-3 * max(1.0, dxn.double().norm().item()), (got, want)


# ---- streams, graphs, repeatability ---------------------------------------------------------

def _head_pass(x, gamma, beta, w, t, up, seed=5):
    y, mean, rstd = conv.layer_norm(x, gamma, beta, out_dtype=w.dtype, dropout_p=0.1, seed=seed)
    loss, lse = conv.linear_cross_entropy(y, w, t)
    dy, dw = conv.linear_cross_entropy_backward(up, y, w, t, lse)
    dx, dg, db = conv.layer_norm_backward(dy, x, gamma, mean, rstd, dropout_p=0.1, seed=seed)
    return [loss, lse, dw, dx, dg, db]


def _head_inputs(dt="bf16", N=300, V=2000, D=256):
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(N, D, generator=g, device=DEV)
    w = (torch.randn(V, D, generator=g, device=DEV) * 0.1).to(TYPES[dt])
    t = torch.randint(0, V, (N,), generator=g, device=DEV)
    return x, torch.ones(D, device=DEV), torch.zeros(D, device=DEV), w, t, torch.full((N,), 1.0 / N, device=DEV)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_same_bits_every_time_and_on_another_stream(dt):
    args = _head_inputs(dt)
    first = _head_pass(*args)
    torch.cuda.synchronize()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(_head_pass(*args), first))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = _head_pass(*args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, first))


def test_captured_graph_replays():
    args = _head_inputs()
    want = _head_pass(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _head_pass(*args)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        out = _head_pass(*args)
    for k in range(4):
        for o in out:
            o.zero_()
        if k == 2:                                   # new inputs in the captured buffers
            args[0].mul_(0.5).add_(0.1)
            want = _head_pass(*args)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), f"replay {k}"


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_workspace_contents_are_never_read_before_written(dt):
    x, w, t, up = (v.to(DEV) for v in _xent_case(130, 700, 100, dt, seed=4))
    outs = []
    for fill in (0, 255):
        n = conv.linear_cross_entropy_workspace_size(x, w, backward=True)
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        loss, lse = torch.empty(130, device=DEV), torch.empty(130, device=DEV)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        conv.linear_cross_entropy_into(x, w, t, loss, lse, ws)
        ws.fill_(fill)
        conv.linear_cross_entropy_backward_into(up, x, w, t, lse, dx, dw, ws)
        outs.append([loss, lse, dx, dw])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_example_head_learns(dt):
    """The example's head on frozen convolution features: the held-out loss falls
    from about log(classes) well below it."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, before, after = mod.train(steps=60, classes=200, dtype=TYPES[dt])
    _say(f"example {dt}: {before:.3f} -> {after:.3f}, last steps {losses[-3:]}")
    assert all(np.isfinite(losses)) and before > 4.0 and after < 0.5 * before


def test_python_refusals():
    x = torch.zeros(4, 8, device=DEV)
    w = torch.zeros(5, 8, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    v = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError, match="target"):
        conv.linear_cross_entropy(x, w, t.int())
    with pytest.raises(ValueError, match="target"):
        conv.linear_cross_entropy(x, w, t[:3])
    with pytest.raises(ValueError, match="ws"):
        conv.linear_cross_entropy_into(x, w, t, v, v.clone(), torch.empty(1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="dx"):
        conv.linear_cross_entropy_backward_into(v, x, w, t, v, x.half(), w, None)
    with pytest.raises(ValueError, match="weight"):
        conv.layer_norm(x, torch.ones(7, device=DEV))
    with pytest.raises(ValueError, match="dweight|weight"):
        conv.layer_norm(x, torch.ones(8, device=DEV).half())
    with pytest.raises(conv.Conv2dError, match="UNSUPPORTED"):
        conv.layer_norm(x.half(), out_dtype=torch.float32)
    with pytest.raises(conv.Conv2dError, match="INVALID"):
        conv.dropout(x, 1.5, 0)
    with pytest.raises(ValueError, match="y must be"):
        conv.dropout_into(x, x.half(), 0.5, 0)
