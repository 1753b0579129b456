"""Block operators without a GPU: the header against the binding, the oracle's
gradients against differences, the levels of 8-bit states, refusals of bad
descriptors and arguments, workspace sizes, and the device that calls are made on."""
import contextlib
import ctypes
import os
import re
import subprocess

import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _block, _lib, block, head
from oracle import block as ref
from test_head_binding_host import DeviceTensor
from test_head_host import _differences

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN, INF = float("nan"), float("inf")
P = 4096            # any non-NULL, aligned address: refused calls never touch it


def test_header_matches_binding_and_library():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "im2win_block.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b([a-z0-9_]+)\s*\([^;{]*\)\s*;", text)))
    assert declared == sorted(_block.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIBPATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(_block.EXPORTS) <= exported
    for name, code in _block.ACTIVATIONS.items():
        assert re.search(rf"\bFF_{name.upper()} = {code}\b", text)
    for name, code in _block.KINDS.items():
        assert re.search(rf"\bRN_{name.upper()} = {code}\b", text)


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"feed_forward_desc_t": _block.FeedForwardDesc, "residual_norm_desc_t": _block.ResidualNormDesc,
               "adamw_tensor_t": _block.AdamWTensor, "adamw_desc_t": _block.AdamWDesc}
    lines = [f'printf("%zu ", sizeof({n}));' for n in structs]
    for n, t in structs.items():
        lines += [f'printf("%zu ", offsetof({n}, {f}));' for f, _ in t._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "im2win_block.h"\nint main(void) {' +
                   "\n".join(lines) + "return 0; }")
    exe = tmp_path / "s"
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = [ctypes.sizeof(t) for t in structs.values()]
    want += [getattr(t, f).offset for t in structs.values() for f, _ in t._fields_]
    assert got == want


# ---- the oracle against differences ---------------------------------------------------

@pytest.mark.parametrize("act", sorted(_block.ACTIVATIONS))
def test_oracle_feed_forward_gradient_against_differences(act):
    g = torch.Generator().manual_seed(3)
    x, wg, wu, wd = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((4, 3), (5, 3), (5, 3), (2, 5)))
    dy = torch.randn(4, 2, generator=g, dtype=torch.float64)

    def f():
        return (ref.feed_forward(x, wg, wu, wd, act)[0] * dy).sum().item()
    got = ref.feed_forward_grad(dy, x, wg, wu, wd, act)[:4]
    for a, v in zip(got, (x, wg, wu, wd)):
        assert torch.allclose(a, _differences(f, v), rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [True, False])
def test_oracle_residual_norm_gradient_against_differences(kind, post):
    g = torch.Generator().manual_seed(4)

    def rnd(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)
    b, r, gate, pw, pb, w, bias, dy, dout = (rnd(6, 5), rnd(6, 5), rnd(3, 5), rnd(5), rnd(5), rnd(5), rnd(5), rnd(6, 5),
                                             rnd(6, 5))
    rs, bs = 0.75, 1.25
    if not post:
        pw = pb = None

    def f():
        out, y, _, _ = ref.residual_norm(b, r, gate, pw, pb, w, bias, kind, post, 1e-5, rs, bs)
        return ((y * dy).sum() + (out * dout).sum()).item()
    out, _, st, _ = ref.residual_norm(b, r, gate, pw, pb, w, bias, kind, post, 1e-5, rs, bs)
    got = ref.residual_norm_grad(dy, dout, b, out, st, gate, pw, pb, w, kind, post, rs, bs)
    wrt = {"dr": r, "db": b, "gate": gate, "weight": w, "bias": bias}
    if post:
        wrt.update(post_weight=pw, post_bias=pb)
    for name, v in wrt.items():
        assert torch.allclose(got[name], _differences(f, v), rtol=1e-6, atol=1e-7), name


def test_codes_have_the_values_mean():
    """Over all 65536 numbers a value's mean code value is the value, to the share of one
    number; levels themselves keep their code."""
    u = torch.arange(65536)
    for power, top in ((2, 127), (4, 255)):
        for x in (0.3, 1.0, 2.5, 7.0 ** power + 0.125, (top - 0.5) ** power, float(top ** power)):
            k = ref.code(torch.full((65536,), x, dtype=torch.float64), u, power, top)
            c = int(x ** (1.0 / power) + 1e-12)
            width = (c + 1) ** power - c ** power
            assert abs((k ** power).mean().item() - x) <= width / 65536 + 1e-6 * x
            if abs(x - c ** power) < 1e-9:
                assert bool((k == c).all())


def test_oracle_numbers_follow_the_definition():
    um, uv = ref.numbers(6, 9, (3 << 32) + 5, 0x123456789ABCDEF0)
    for i in range(9):
        e = 6 + i
        w = ref.philox4x32((e // 4, 0, 5, 3), (0x9ABCDEF0, 0x12345678))[e % 4]
        assert um[i] == w & 0xFFFF and uv[i] == w >> 16


# ---- refusals of the C entry points ------------------------------------------------------

def _status(name, desc, *args):
    return getattr(_block.lib(), name)(ctypes.byref(desc), *args)


FF = dict(N=4, D=16, F=24, O=8, ldx=0, ldg=0, ldu=0, ldd=0, ldy=0, dtype=1, act=0, reserved=0, reserved2=0)


@pytest.mark.parametrize("bad,want", [
    (dict(N=-1), 1), (dict(N=(1 << 22) + 1), 1), (dict(D=0), 1), (dict(F=0), 1), (dict(O=0), 1),
    (dict(D=(1 << 20) + 1), 1), (dict(F=(1 << 20) + 1), 1), (dict(O=(1 << 20) + 1), 1), (dict(ldx=15), 1),
    (dict(ldg=15), 1), (dict(ldu=15), 1), (dict(ldd=23), 1), (dict(ldy=7), 1), (dict(ldx=(1 << 20) + 8), 1),
    (dict(reserved=1), 1), (dict(reserved2=1), 1), (dict(dtype=3), 4), (dict(dtype=-1), 4), (dict(act=5), 4),
    (dict(act=-1), 4),
])
def test_feed_forward_refuses(bad, want):
    d = _block.FeedForwardDesc(**{**FF, **bad})
    assert _status("feed_forward_fwd", d, P, P, P, P, P, P, P, None) == want
    assert _status("feed_forward_bwd", d, *[P] * 11, None) == want
    assert _status("feed_forward_saved_size", d) == 0 and _status("feed_forward_bwd_workspace_size", d) == 0
    assert _status("feed_forward_fwd_workspace_size", d, 1) == 0


def test_feed_forward_pointers():
    d = _block.FeedForwardDesc(**FF)
    assert _block.lib().feed_forward_fwd(None, *[P] * 7, None) == 2
    for i in range(5):
        a = [P] * 7
        a[i] = None
        assert _status("feed_forward_fwd", d, *a, None) == 2, i
        a[i] = P + 8 if i < 4 else P + 1        # rows of whole granules; y any element
        assert _status("feed_forward_fwd", d, *a, None) == 3, i
    assert _status("feed_forward_fwd", d, *[P] * 5, None, None, None) == 5
    assert _status("feed_forward_fwd", d, *[P] * 5, P + 16, P, None) == 3
    assert _status("feed_forward_fwd", d, *[P] * 6, P + 16, None) == 3
    for i in range(10):
        a = [P] * 11
        a[i] = None
        assert _status("feed_forward_bwd", d, *a, None) == 2, i
        a[i] = P + (16 if i == 5 else 8 if i < 5 else 1)
        assert _status("feed_forward_bwd", d, *a, None) == 3, i
    assert _status("feed_forward_bwd", d, *[P] * 10, None, None) == 5
    # rows that are no whole granules start at any element
    odd = _block.FeedForwardDesc(**{**FF, "D": 15})
    assert _status("feed_forward_fwd", odd, P + 2, P + 2, P + 2, P, P, P, P + 16, None) == 3
    assert _status("feed_forward_fwd", odd, P + 1, P, P, P, P, P, P, None) == 3


RN = dict(N=6, C=16, groups=3, ldb=0, ldr=0, ldo=0, ldy=0, lddr=0, lddb=0, lddo=0, lddy=0, dtype=0, branch_dtype=2, kind=0,
          post=1, eps=1e-5, residual_scale=1.0, branch_scale=1.0)


@pytest.mark.parametrize("bad,want", [
    (dict(N=-1), 1), (dict(N=1 << 31), 1), (dict(C=0), 1), (dict(C=1 << 27), 1), (dict(groups=-1), 1), (dict(groups=4), 1),
    (dict(groups=12), 1), (dict(ldb=15), 1), (dict(ldr=15), 1), (dict(ldo=15), 1), (dict(ldy=15), 1), (dict(lddr=15), 1),
    (dict(lddb=15), 1), (dict(lddo=15), 1), (dict(lddy=15), 1), (dict(N=1 << 30, groups=1, ldb=1 << 20), 1),
    (dict(post=2), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(residual_scale=INF), 1), (dict(branch_scale=NAN), 1),
    (dict(residual_scale=1e39), 1), (dict(branch_scale=-1e39), 1), (dict(eps=1e39), 1),
    (dict(dtype=5), 4), (dict(branch_dtype=7), 4), (dict(dtype=1), 4), (dict(dtype=2, branch_dtype=0), 4), (dict(kind=2), 4),
])
def test_residual_norm_refuses(bad, want):
    d = _block.ResidualNormDesc(**{**RN, **bad})
    assert _status("residual_norm_fwd", d, *[P] * 10, None) == want
    assert _status("residual_norm_bwd", d, *[P] * 17, None) == want
    assert _status("residual_norm_bwd_workspace_size", d) == 0


def test_residual_norm_pointers():
    d = _block.ResidualNormDesc(**RN)
    for i in (0, 1, 2, 7, 8):                           # b, r, gate, out, y
        a = [P] * 10
        a[i] = None
        assert _status("residual_norm_fwd", d, *a, None) == 2, i
        a[i] = P + 1
        assert _status("residual_norm_fwd", d, *a, None) == 3, i
    assert _status("residual_norm_fwd", d, *[P] * 9, P + 8, None) == 3          # stats
    for i in (0, 2, 3, 4, 5, 9, 10):                    # dy, b, out, stats, gate, dr, db
        a = [P] * 17
        a[i] = None
        assert _status("residual_norm_bwd", d, *a, None) == 2, i
        a[i] = P + (8 if i == 4 else 1)
        assert _status("residual_norm_bwd", d, *a, None) == 3, i
    assert _status("residual_norm_bwd", d, *[P] * 16, None, None) == 5
    assert _status("residual_norm_bwd", d, *[P] * 16, P + 16, None) == 3
    plain = _block.ResidualNormDesc(**{**RN, "post": 0, "groups": 0})
    assert _status("residual_norm_fwd", plain, P, P, None, P, None, P, P, P, P, P, None) == 1   # no norm, no weight of it
    assert _status("residual_norm_fwd", plain, P, P, P, None, None, P, P, P, P, P, None) == 2   # a gate without groups
    a = [P, P, P, P, P, None, None, None, P, P, P, P, None, None, P, P, P]
    assert _status("residual_norm_bwd", plain, *a, None) == 1                   # dgate without a gate
    a[11], a[12] = None, P
    assert _status("residual_norm_bwd", plain, *a, None) == 1                   # dpost_weight without its norm


ADAM = dict(count=1, bits=8, reserved=0, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, seed=0, step=1)
TENSOR = dict(param=P, grad=P, copy=P, m=P, v=P, m_scale=P, v_scale=P, n=300, first=256, param_dtype=0, grad_dtype=1,
              copy_dtype=2, reserved=0, lr=1e-3, weight_decay=0.1)


def _adam(desc=(), tensor=(), pointers=(None, None, None)):
    t = _block.AdamWTensor(**{**TENSOR, **dict(tensor)})
    return _status("adamw_step", _block.AdamWDesc(**{**ADAM, **dict(desc)}), ctypes.byref(t), *pointers, None)


@pytest.mark.parametrize("bad,want", [
    (dict(count=-1), 1), (dict(reserved=1), 1), (dict(beta1=1.0), 1), (dict(beta1=-0.1), 1), (dict(beta2=1.0), 1),
    (dict(beta2=NAN), 1), (dict(eps=-1.0), 1), (dict(eps=INF), 1), (dict(grad_scale=NAN), 1), (dict(step=0), 1),
    (dict(step=-3), 1), (dict(eps=1e39), 1), (dict(grad_scale=-1e39), 1), (dict(bits=16), 4), (dict(bits=0), 4),
])
def test_adamw_refuses(bad, want):
    assert _adam(bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), 1), (dict(n=1 << 41), 1), (dict(reserved=1), 1), (dict(lr=NAN), 1), (dict(weight_decay=INF), 1),
    (dict(first=-256), 1), (dict(first=100), 1), (dict(first=1 << 62 | 256), 1), (dict(lr=1e39), 1), (dict(weight_decay=-1e39), 1), (dict(param_dtype=3), 4), (dict(grad_dtype=-1), 4), (dict(copy_dtype=9), 4),
    (dict(param=None), 2), (dict(grad=None), 2), (dict(m=None), 2), (dict(v=None), 2), (dict(m_scale=None), 2),
    (dict(v_scale=None), 2), (dict(param=P + 2), 3), (dict(grad=P + 1), 3), (dict(copy=P + 1), 3), (dict(m=P + 2), 3),
    (dict(v=P + 2), 3), (dict(m_scale=P + 2), 3), (dict(v_scale=P + 1), 3),
])
def test_adamw_refuses_tensors(bad, want):
    assert _adam(tensor=bad) == want


def test_adamw_pointers():
    assert _status("adamw_step", _block.AdamWDesc(**ADAM), None, None, None, None, None) == 2
    assert _adam(pointers=(P, None, None)) == 1                 # two steps
    assert _adam(dict(step=0), pointers=(P + 4, None, None)) == 3
    assert _adam(pointers=(None, P + 2, None)) == 3 and _adam(pointers=(None, None, P + 2)) == 3
    assert _adam(dict(bits=32)) == 1                            # scales and a number with 32 bits
    assert _adam(dict(bits=32), dict(m_scale=None, v_scale=None, first=0, n=0)) == 0
    assert _adam(dict(count=0)) == 0
    L = _block.lib()
    assert L.adamw_values(-1, P, P, P, P, P, P, None) == 1 and L.adamw_values(4, P, None, P, P, P, P, None) == 2
    assert L.adamw_values(4, P + 1, P, P, P, P, P, None) == 3 and L.adamw_values(4, P, P, P, P, P + 2, P, None) == 3
    assert L.adamw_values(0, None, None, None, None, None, None, None) == 0


def test_workspaces_stay_bounded():
    """A training pass keeps 8 bytes (fp32 factors) and its type's 2 of h per row and hidden
    feature, the backward workspace the 4 of da and du: no slabs beside large products."""
    d = _block.FeedForwardDesc(8192, 4096, 16384, 4096, 0, 0, 0, 0, 0, _lib.BF16, 0, 0, 0)
    nf = 8192 * 16384
    assert _block.size("feed_forward_saved_size", d) == nf * 10
    assert _block.size("feed_forward_bwd_workspace_size", d) <= nf * 4 + 4096
    assert _block.size("feed_forward_fwd_workspace_size", d, 1) == 0
    assert _block.size("feed_forward_fwd_workspace_size", d, 0) == nf * 2
    one = _block.FeedForwardDesc(1, 4096, 8192, 4096, 0, 0, 0, 0, 0, _lib.BF16, 0, 0, 0)
    assert _block.size("feed_forward_fwd_workspace_size", one, 0) <= 8192 * 4 + 512


# ---- refusals of the Python entry points, and the device of a call ------------------------------

def test_python_checks_name_the_argument():
    x, w = torch.zeros(4, 8), torch.zeros(5, 8)
    for f in (lambda: conv.feed_forward(x, w, w, w.t()), lambda: conv.residual_norm(x, x),
              lambda: conv.adamw_state([x]), lambda: conv.feed_forward_workspace_size(x, w, w, w)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    a, v = DeviceTensor(4, 8), DeviceTensor(5, 8)
    d = DeviceTensor(6, 5)
    for args, what in (((a, v, v, DeviceTensor(6, 4)), r"w_down \[O\]\[F\]"), ((a, DeviceTensor(5, 7), v, d), "w_gate"),
                       ((a, v, DeviceTensor(4, 8), d), "w_up"),
                       ((a, v, DeviceTensor(5, 8, dtype=torch.float16), d), "w_up")):
        with pytest.raises(ValueError, match=what):
            conv.feed_forward_workspace_size(*args)
    with pytest.raises(ValueError, match="activation"):
        conv.feed_forward_into(a, v, v, d, DeviceTensor(4, 6), None, None, activation="tanh")
    with pytest.raises(ValueError, match="y and dy"):
        conv.feed_forward_into(a, v, v, d, DeviceTensor(4, 5), None, None)
    with pytest.raises(ValueError, match="kind"):
        conv.residual_norm_into(a, a, a, a, None, kind="batch")
    with pytest.raises(ValueError, match="groups"):
        conv.residual_norm_into(a, a, a, a, None, gate=DeviceTensor(3, 8))
    with pytest.raises(ValueError, match="post_weight"):
        conv.residual_norm_into(a, a, a, a, None, post=False, post_weight=DeviceTensor(8))
    with pytest.raises(ValueError, match="dgate"):
        conv.residual_norm_backward_into(a, None, a, a, DeviceTensor(4, 4), a, a, None, dgate=DeviceTensor(8))
    with pytest.raises(ValueError, match="bits"):
        conv.AdamWState([4], 16, "cpu")


def _calls():
    x, w, wd, v4 = DeviceTensor(4, 8), DeviceTensor(8, 8), DeviceTensor(8, 8), DeviceTensor(4, 4)
    ws = DeviceTensor(1 << 20, dtype=torch.uint8)
    state = conv.AdamWState([32, 300], 8, "cpu")
    for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        t = getattr(state, name)
        setattr(state, name, DeviceTensor(*t.shape, dtype=t.dtype))
    p = [DeviceTensor(4, 8), DeviceTensor(300)]
    n = state.exp_avg.numel()
    return {
        "feed_forward_fwd": lambda: block.feed_forward_into(x, w, w, wd, x, None, ws),
        "feed_forward_bwd": lambda: block.feed_forward_backward_into(x, x, w, w, wd, ws, x, w, w, wd, ws),
        "residual_norm_fwd": lambda: block.residual_norm_into(x, x, x, x, v4),
        "residual_norm_bwd": lambda: block.residual_norm_backward_into(x, x, x, x, v4, x, x, ws),
        "adamw_step": lambda: block.adamw(p, p, state, 3, 1e-3),
        "adamw_values": lambda: block.adamw_state_values_into(state, DeviceTensor(n), DeviceTensor(n)),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
@pytest.mark.parametrize("current", [0, 1])
def test_calls_are_made_on_the_tensors_device(monkeypatch, name, current):
    head._torch_names()
    state = {"device": current}
    seen = []

    @contextlib.contextmanager
    def guard(dev):
        before, state["device"] = state["device"], dev
        yield
        state["device"] = before
    monkeypatch.setattr(head, "_current_device", lambda: state["device"], raising=False)
    monkeypatch.setattr(head, "_device_guard", guard, raising=False)
    monkeypatch.setattr(head, "_raw_stream", lambda dev: ("stream of", dev))
    monkeypatch.setattr(_block, "call", lambda name, *args: seen.append((name, state["device"], args[-1])))
    _calls()[name]()
    assert seen == [(name, 1, ("stream of", 1))] and state["device"] == current


def test_the_optimizers_table(monkeypatch):
    """What adamw hands to the library, entry by entry, after the state's buffers moved."""
    head._torch_names()
    monkeypatch.setattr(head, "_current_device", lambda: 1, raising=False)
    monkeypatch.setattr(head, "_raw_stream", lambda dev: 7)
    calls = []
    monkeypatch.setattr(_block, "call", lambda name, d, t, *rest: calls.append((d, list(t), rest)))
    for bits in (32, 8, 8):
        state = conv.AdamWState([32, 300, 1], bits, "cpu")
        names = ("exp_avg", "exp_avg_sq") + (("exp_avg_scale", "exp_avg_sq_scale") if bits == 8 else ())
        for _ in range(2):
            for name in names:
                t = getattr(state, name)
                setattr(state, name, DeviceTensor(*t.shape, dtype=t.dtype))
            p = [DeviceTensor(4, 8), DeviceTensor(300, dtype=torch.bfloat16), DeviceTensor(1)]
            g = [DeviceTensor(32, dtype=torch.float16), DeviceTensor(300), DeviceTensor(1)]
            c = [None, DeviceTensor(300, dtype=torch.float16), None]
            conv.adamw(p, g, state, 9, [1.0, 2.0, 3.0], weight_decay=0.5, copies=c, seed=11)
            d, table, rest = calls.pop()
            assert (d.count, d.bits, d.step, d.seed, rest) == (3, bits, 9, 11, (None, None, None, 7))
            es = 1 if bits == 8 else 4
            for i, (e, at, n) in enumerate(zip(table, (0, 256, 768), (32, 300, 1))):
                assert (e.param, e.grad, e.n, e.lr, e.weight_decay) == (p[i].data_ptr(), g[i].data_ptr(), n, i + 1.0, 0.5)
                assert (e.m, e.v) == (state.exp_avg.data_ptr() + at * es, state.exp_avg_sq.data_ptr() + at * es)
                assert (e.param_dtype, e.grad_dtype) == ((0, 1), (2, 0), (0, 0))[i] and e.reserved == 0
                assert (e.copy, e.copy_dtype) == ((c[1].data_ptr(), 1) if i == 1 else (None, 0))
                if bits == 8:
                    assert (e.first, e.m_scale) == (at, state.exp_avg_scale.data_ptr() + at // 256 * 4)
                    assert e.v_scale == state.exp_avg_sq_scale.data_ptr() + at // 256 * 4
                else:
                    assert (e.first, e.m_scale, e.v_scale) == (0, None, None)
    for bad, what in ((dict(params=p[:2]), "number"), (dict(copies=c[:2]), "copies"), (dict(step=0), "from 1 on"),
                      (dict(lr=[1.0, 2.0]), "lr"), (dict(grads=[g[0], g[1], DeviceTensor(2)]), r"grads\[2\]"),
                      (dict(grads=[g[0], None, g[2]]), r"grads\[1\] is None")):
        with pytest.raises(ValueError, match=what):
            conv.adamw(**{**dict(params=p, grads=g, state=state, step=9, lr=1.0), **bad})
    # one tensor twice would be updated by two workgroups at once; empty ones share an address
    state, twice = conv.AdamWState([6, 4, 0, 6, 0], 32, "cpu"), DeviceTensor(6)
    for name in ("exp_avg", "exp_avg_sq"):
        setattr(state, name, DeviceTensor(*getattr(state, name).shape))
    p = [twice, DeviceTensor(4), DeviceTensor(0), DeviceTensor(6), DeviceTensor(0)]
    g = [DeviceTensor(n) for n in state.sizes]
    p[2].data_ptr = p[4].data_ptr = lambda: 0
    conv.adamw(p, g, state, 1, 1.0)
    with pytest.raises(ValueError, match=r"params\[3\] is in the list twice"):
        conv.adamw(p[:3] + [twice] + p[4:], g, state, 1, 1.0)
    with pytest.raises(ValueError, match=r"copies\[3\] is in the list twice"):
        conv.adamw(p, g, state, 1, 1.0, copies=[g[0], None, None, g[0], None])


def test_rows_of_blocks_have_records_of_their_own():
    """The backward norm's records (block + group) are never shared and leave no gap."""
    for N, G, B in ((12, 3, 5), (7, 7, 7), (30, 2, 11), (64, 64, 10), (100, 4, 25), (256, 1, 256), (21, 3, 7)):
        rows, q, rem = N // G, N // B, N % B
        first = [q * b + min(b, rem) for b in range(B + 1)]
        seen = []
        for b in range(B):
            at = first[b]
            while at < first[b + 1]:
                g = at // rows if G > 1 else 0
                to = min(first[b + 1], (g + 1) * rows) if G > 1 else first[b + 1]
                seen.append(b + g)
                if to == first[b + 1] and G > 1 and to % rows == 0 and to < N:
                    seen.append(b + g + 1)
                at = to
        assert sorted(seen) == list(range(B + G - 1))
