"""Training-head operators without a GPU: the header against the binding, the
oracle's generator against published values, its gradients against
differences, refusals of bad descriptors, and workspace sizes."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _head, _lib
from oracle import head as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAN = float("nan")


def test_header_matches_binding_and_library():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "im2win_head.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b([a-z0-9_]+)\s*\([^;{]*\)\s*;", text)))
    assert declared == sorted(_head.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIBPATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(_head.EXPORTS) <= exported


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "im2win_head.h"\nint main(void) { printf("%zu %zu %zu", '
                   'sizeof(dropout_desc_t), sizeof(layer_norm_desc_t), sizeof(linear_xent_desc_t)); return 0; }')
    exe = tmp_path / "s"
    subprocess.run(["gcc", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(t) for t in (_head.DropoutDesc, _head.LayerNormDesc, _head.LinearXentDesc)]


@pytest.mark.parametrize("counter,key,want", [
    # the known answers published with the generator (philox4x32, 10 rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_known_answers(counter, key, want):
    assert tuple(ref.philox4x32(counter, key)) == want


def test_element_numbers_follow_the_definition():
    seed, offset = 0x123456789ABCDEF0, (1 << 32) - 2
    got = ref.numbers(5, 40, seed, offset)
    for i, u in zip(range(5, 45), got):
        b = offset + i // 8
        w = ref.philox4x32((b & 0xFFFFFFFF, b >> 32, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))[(i % 8) // 2]
        assert u == ((w >> 16) if i % 2 else (w & 0xFFFF))


def test_drop_rate_and_independence_of_neighbours():
    u = ref.numbers(0, 1 << 18, 7, 0)
    for p in (0.1, 0.5):
        drop = (u < p * 65536).astype(np.float64)
        n = drop.size
        # six standard deviations of a binomial share, and of the products of neighbours
        assert abs(drop.mean() - p) < 6 * np.sqrt(p * (1 - p) / n)
        for lag in (1, 2, 4, 8):
            pair = (drop[lag:] - p) * (drop[:-lag] - p)
            assert abs(pair.mean()) < 6 * p * (1 - p) / np.sqrt(pair.size)


def _differences(f, x, h=1e-6):
    g = torch.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        out[i] = (up - f()) / (2 * h)
        flat[i] = keep
    return g


def test_oracle_layer_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    for dim, shape in ((1, (3, 5)), (1, (2, 4, 3))):
        x = torch.randn(shape, generator=g, dtype=torch.float64)
        C = shape[dim]
        w, b = torch.randn(C, generator=g, dtype=torch.float64), torch.randn(C, generator=g, dtype=torch.float64)
        dy = torch.randn(shape, generator=g, dtype=torch.float64)
        drop = ref.drop_factors(shape, 0.25, 9)

        def f():
            return (ref.layer_norm(x, w, b, 1e-5, dim)[0] * drop * dy).sum().item()
        _, mean, rstd = ref.layer_norm(x, w, b, 1e-5, dim)
        got = ref.layer_norm_grad(dy * drop, x, w, mean, rstd, dim)
        # central differences of step 1e-6 in 64 bits: truncation 1e-12, rounding 1e-10 relative to the terms
        for a, v in zip(got, (x, w, b)):
            assert torch.allclose(a, _differences(f, v), rtol=1e-6, atol=1e-7)


def test_oracle_cross_entropy_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((4, 3), generator=g, dtype=torch.float64)
    w = torch.randn((6, 3), generator=g, dtype=torch.float64)
    t = torch.tensor([0, 5, -1, 6])
    up = torch.randn(4, generator=g, dtype=torch.float64)

    def f():
        return (ref.cross_entropy(x, w, t)[0] * up).sum().item()
    dx, dw, _ = ref.cross_entropy_grad(up, x, w, t)
    assert torch.allclose(dx, _differences(f, x), rtol=1e-6, atol=1e-7)
    assert torch.allclose(dw, _differences(f, w), rtol=1e-6, atol=1e-7)
    loss, lse = ref.cross_entropy(x, w, t)
    assert loss[2] == 0 and lse[3] == 0 and not dx[2:].any()


P = 4096            # any non-NULL, aligned address: refused calls never touch it


def _status(name, desc, *args):
    return getattr(_head.lib(), name)(ctypes.byref(desc), *args)


@pytest.mark.parametrize("bad,want", [
    (dict(n=-1), 1), (dict(n=1 << 41), 1), (dict(reserved=1), 1), (dict(p=-0.1), 1), (dict(p=1.5), 1), (dict(p=NAN), 1),
    (dict(dtype=3), 4), (dict(dtype=-1), 4),
])
def test_dropout_refuses(bad, want):
    f = dict(n=16, dtype=0, reserved=0, p=0.5, seed=1, offset=0)
    f.update(bad)
    assert _status("dropout_fwd", _head.DropoutDesc(**f), P, P, None) == want


def test_dropout_pointers():
    d = _head.DropoutDesc(16, 0, 0, 0.5, 1, 0)
    assert _status("dropout_fwd", d, None, P, None) == 2
    assert _status("dropout_fwd", d, P, None, None) == 2
    assert _status("dropout_fwd", d, P + 2, P, None) == 3
    assert _head.lib().dropout_fwd(None, P, P, None) == 2
    assert _status("dropout_fwd", _head.DropoutDesc(0, 0, 0, 0.5, 1, 0), None, None, None) == 0


NORM = dict(N=4, C=8, P=1, ldx=0, ldy=0, lddx=0, dtype=1, y_dtype=1, layout=1, reserved=0, eps=1e-5, dropout_p=0.0,
            seed=0, offset=0)


@pytest.mark.parametrize("bad,want", [
    (dict(N=-1), 1), (dict(C=0), 1), (dict(P=0), 1), (dict(P=2), 1), (dict(ldx=7), 1), (dict(ldy=7), 1),
    (dict(lddx=7), 1), (dict(N=1 << 30, C=1 << 20), 1), (dict(N=1 << 31), 1), (dict(C=1 << 27), 1),
    (dict(reserved=1), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(dropout_p=1.1), 1), (dict(dropout_p=NAN), 1),
    (dict(dtype=5), 4), (dict(y_dtype=5), 4), (dict(layout=2), 4), (dict(y_dtype=0), 4), (dict(y_dtype=2), 4),
    (dict(layout=0, ldx=8), 1), (dict(layout=0, P=1 << 30, N=1 << 12), 1),
])
def test_layer_norm_refuses(bad, want):
    d = _head.LayerNormDesc(**{**NORM, **bad})
    assert _status("layer_norm_fwd", d, P, P, P, P, P, P, None) == want
    assert _status("layer_norm_bwd", d, P, P, P, P, P, P, P, P, P, None) == want
    assert _status("layer_norm_bwd_workspace_size", d) == 0


def test_layer_norm_pointers():
    d = _head.LayerNormDesc(**NORM)
    assert _status("layer_norm_fwd", d, None, P, P, P, P, P, None) == 2
    assert _status("layer_norm_fwd", d, P, P, P, None, P, P, None) == 2
    assert _status("layer_norm_fwd", d, P, P, P, P, P, None, None) == 2       # mean without rstd
    assert _status("layer_norm_fwd", d, P + 1, P, P, P, P, P, None) == 3
    assert _status("layer_norm_fwd", d, P, P + 2, P, P, P, P, None) == 3
    ok = [P] * 9
    for i in (0, 1, 3, 4, 5, 6, 7):
        a = list(ok)
        a[i] = None
        assert _status("layer_norm_bwd", d, *a, None) == 2, i
    assert _status("layer_norm_bwd", d, *ok[:8], None, None) == 5
    assert _status("layer_norm_bwd", d, *ok[:8], P + 16, None) == 3
    assert _status("layer_norm_bwd_workspace_size", d) >= 2 * 8 * 4


XENT = dict(N=4, V=10, D=8, ldx=0, ldw=0, dtype=1, reserved=0)


@pytest.mark.parametrize("bad,want", [
    (dict(N=-1), 1), (dict(V=0), 1), (dict(D=0), 1), (dict(ldx=7), 1), (dict(ldw=7), 1), (dict(reserved=2), 1),
    (dict(N=(1 << 22) + 1), 1), (dict(V=(1 << 24) + 1), 1), (dict(D=(1 << 20) + 1), 1), (dict(ldx=(1 << 22) + 1), 1),
    (dict(ldw=(1 << 20) + 1), 1), (dict(dtype=3), 4),
])
def test_linear_xent_refuses(bad, want):
    d = _head.LinearXentDesc(**{**XENT, **bad})
    assert _status("linear_xent_fwd", d, P, P, P, P, P, P, None) == want
    assert _status("linear_xent_bwd", d, P, P, P, P, P, P, P, P, None) == want
    assert _status("linear_xent_fwd_workspace_size", d) == 0
    assert _status("linear_xent_bwd_workspace_size", d) == 0


def test_linear_xent_pointers():
    d = _head.LinearXentDesc(**XENT)
    ok = [P] * 6
    for i in range(5):
        a = list(ok)
        a[i] = None
        assert _status("linear_xent_fwd", d, *a, None) == 2, i
    assert _status("linear_xent_fwd", d, P, P, P + 4, P, P, P, None) == 3
    # rows of whole 16-byte granules start on a 16-byte boundary
    assert _status("linear_xent_fwd", d, P + 8, P, P, P, P, P, None) == 3
    assert _status("linear_xent_fwd", d, P, P + 8, P, P, P, P, None) == 3
    assert _status("linear_xent_bwd", d, P, P, P + 8, P, P, P, P, P, None) == 3
    assert _status("linear_xent_fwd", _head.LinearXentDesc(**{**XENT, "D": 7}), P, P + 1, P, P, P, P, None) == 3
    ok = [P] * 8
    for i in range(7):
        a = list(ok)
        a[i] = None
        assert _status("linear_xent_bwd", d, *a, None) == 2, i
    assert _status("linear_xent_bwd_workspace_size", d) > 0
    assert _status("linear_xent_bwd", d, *ok[:7], None, None) == 5
    assert _status("linear_xent_bwd", d, *ok[:7], P + 8, None) == 3


def test_python_checks_name_the_argument():
    x = torch.zeros(4, 8)
    for f in (lambda: conv.dropout(x, 0.5, 1), lambda: conv.layer_norm(x),
              lambda: conv.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int64))):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(ValueError, match=r"\[V\]\[D\]"):
        conv.linear_cross_entropy_workspace_size(x, torch.zeros(3, 7))
    with pytest.raises(TypeError, match="share a dtype"):
        conv.linear_cross_entropy_workspace_size(x, x.half())
    with pytest.raises(TypeError, match="unsupported dtype"):
        conv.layer_norm_workspace_size(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        conv.layer_norm_workspace_size(x.t())
    with pytest.raises(ValueError, match="layout"):
        conv.layer_norm_workspace_size(x, layout="chwn")


def test_workspaces_stay_bounded():
    """No workspace grows with rows x classes: the logits are never held."""
    d = _head.LinearXentDesc(8192, 131072, 4096, 0, 0, _lib.BF16, 0)
    logits = 8192 * 131072 * 2
    assert _head.size("linear_xent_fwd_workspace_size", d) < logits / 8
    assert _head.size("linear_xent_bwd_workspace_size", d) < logits / 2
