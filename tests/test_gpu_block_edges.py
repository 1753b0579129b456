"""Edges of the block kernels: values at the ends of the types' ranges, rows far apart in
size, saturated activations (the bounds' notation is test_gpu_block.py's)."""
import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _lib
from oracle import block as ref
from test_gpu_block import _scales
from test_gpu_head import DEV

pytestmark = pytest.mark.gpu


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
