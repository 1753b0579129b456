"""The training head's Python entry points without a GPU: which device a call is
made on."""
import contextlib

import pytest
import torch

from cnn_convolution_amd import head


class DeviceTensor:
    """As much of a device tensor as the entry points look at, on device 1."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32):
        self._t = torch.zeros(shape, dtype=dtype)
        self.shape, self.dtype = self._t.shape, dtype

    def get_device(self):
        return 1

    def __getattr__(self, name):
        return getattr(self._t, name)


def _calls():
    x, w, v = DeviceTensor(4, 8), DeviceTensor(5, 8), DeviceTensor(4)
    c, t = DeviceTensor(8), DeviceTensor(4, dtype=torch.int64)
    ws = DeviceTensor(1 << 20, dtype=torch.uint8)
    return {
        "dropout_fwd": lambda: head.dropout_into(x, x, 0.5, 1),
        "layer_norm_fwd": lambda: head.layer_norm_into(x, c, c, x, v, v),
        "layer_norm_bwd": lambda: head.layer_norm_backward_into(x, x, c, v, v, x, c, c, ws),
        "linear_xent_fwd": lambda: head.linear_cross_entropy_into(x, w, t, v, v, ws),
        "linear_xent_bwd": lambda: head.linear_cross_entropy_backward_into(v, x, w, t, v, x, w, ws),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
@pytest.mark.parametrize("current", [0, 1])
def test_calls_are_made_on_the_tensors_device(monkeypatch, name, current):
    """Launches go to the current device and the default streams of all devices are
    the null stream: a call for device 1 is made with device 1 current, on the
    stream that is current there, and leaves the current device as it was."""
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
    monkeypatch.setattr(head._head, "call", lambda name, desc, *args: seen.append((name, state["device"], args[-1])))
    _calls()[name]()
    assert seen == [(name, 1, ("stream of", 1))] and state["device"] == current
