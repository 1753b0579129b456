"""Edges of the block kernels: values at the ends of the types' ranges, rows far apart in
size, saturated activations (the bounds' notation is test_gpu_block.py's)."""
import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _lib
from oracle import block as ref
from test_gpu_block import _scales
from test_gpu_head import DEV, U, _close

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    _lib.lib()


# ---- AdamW -----------------------------------------------------------------------------

def _codes_follow(state, m, v, t, seed):
    mk, vk, _, _ = ref.encode(m, v, 0, t, seed, _scales(state, 0))
    assert torch.equal(state.exp_avg[:m.numel()].cpu(), mk), "m codes"
    assert torch.equal(state.exp_avg_sq[:v.numel()].cpu(), vk), "v codes"


def test_adamw_8_bit_scales_above_2_126():
    """Scales whose reciprocal is no normal number: v of gradients around 4e20 (beyond 5.8e20
    v is infinite), m from a restored state."""
    gen = torch.Generator().manual_seed(8)
    n = 700
    g = 10.0 ** (16 + 4.7 * torch.rand(n, generator=gen)) * torch.sign(torch.randn(n, generator=gen))
    g[3], g[400] = 5.5e20, -4e20
    p = torch.zeros(n, device=DEV)
    state = conv.adamw_state([p], 8)
    conv.adamw([p], [g.to(DEV)], state, 1, 1e-3, seed=5)
    assert bool((state.exp_avg_sq_scale[:2] > 2.0 ** 126).all())
    _codes_follow(state, 0.0 + (1 - 0.9) * g.double(), (1 - 0.999) * g.double() ** 2, 1, 5)
    assert all(int(c.max()) == 255 for c in state.exp_avg_sq[:n].split(256))     # the largest v is the scale itself
    state.exp_avg[:n] = torch.randint(-127, 128, (n,), generator=gen).to(torch.int8).to(DEV)
    state.exp_avg_scale.fill_(3e38)
    state.exp_avg_sq_scale.fill_(1.0)
    m0, v0 = ref.decode(*(t.cpu() for t in (state.exp_avg[:n], state.exp_avg_sq[:n], state.exp_avg_scale,
                                            state.exp_avg_sq_scale)))
    conv.adamw([p], [torch.zeros(n, device=DEV)], state, 2, 0.0, seed=6)
    assert bool((state.exp_avg_scale[:3] > 2.0 ** 126).all())
    _codes_follow(state, 0.9 * m0, 0.999 * v0, 2, 6)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("steps", [17.5, 3.5, 1000.5])
def test_adamw_decay_keeps_its_digits(bits, steps):
    """lr * weight_decay of a few and a half of fp32's steps below 1: p (1 - lr weight_decay) is
    rounded once, and the rates and their product to fp32."""
    p = 0.1 * torch.randn(100000, generator=torch.Generator().manual_seed(2))
    q = p.to(DEV)
    lr, decay = 1e-3, steps * 2.0 ** -24 / 1e-3
    conv.adamw([q], [torch.zeros_like(q)], conv.adamw_state([q], bits), 1, lr, weight_decay=decay)
    want = p.double() * (1 - lr * decay)
    _close(q, want, 1.001 * U * want.abs() + 5 * U * lr * decay * p.double().abs() + 2.0 ** -149, "p")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_adamw_infinite_parameters_stay(bits, decay):
    """p (1 - lr weight_decay) - step of an infinite p, and the others as they are without it."""
    gen = torch.Generator().manual_seed(1)
    p, g = torch.randn(300, generator=gen).to(DEV), torch.randn(300, generator=gen).to(DEV)
    q = p.clone()
    q[7], q[261] = INF, -INF
    for t in (p, q):
        conv.adamw([t], [g], conv.adamw_state([t], bits), 1, 1e-2, weight_decay=decay)
    assert q[7] == INF and q[261] == -INF
    p[7], p[261] = INF, -INF
    assert torch.equal(p, q)


def test_adamw_8_bit_denominators_of_denormal_v():
    """A beta2 next to 1 brings a v that is no normal fp32 number up to eps."""
    beta2, eps = 1 - 1e-12, 3e-12
    g = torch.full((300,), 1e-13)
    p = torch.zeros(300, device=DEV)
    conv.adamw([p], [g.to(DEV)], conv.adamw_state([p], 8), 1, 1e-3, beta2=beta2, eps=eps)
    want, m, v = ref.adamw(torch.zeros(300), g, torch.zeros(300), torch.zeros(300), 1, 1e-3, 0.9, beta2, eps, 0.0)
    assert 0 < v.max().item() < 2.0 ** -126
    # v is off by half a subnormal step, 2^-150 of 10^-38 or 2^-23 of it
    _close(p, want, 32 * U * want.abs(), "p")
