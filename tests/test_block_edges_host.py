"""Block operators without a GPU: a process's first call, limits that are refused before
anything is enqueued, workspace sizes, tensors in each other's memory."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import cnn_convolution_amd as conv
from cnn_convolution_amd import _block, _lib, head
from test_head_binding_host import DeviceTensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import os, sys
import torch
from cnn_convolution_amd import _block, _head
import test_block_host, test_head_binding_host
torch._C._cuda_getDevice = lambda: 1
torch._C._cuda_getCurrentRawStream = lambda index: 7
seen = []
_block.call = _head.call = lambda name, *args: seen.append((name, args[-1]))
for calls in (test_block_host._calls(), test_head_binding_host._calls()):
    for name, f in calls.items():
        pid = os.fork()
        if pid == 0:
            try:
                f()
                os._exit(0 if seen == [(name, 7)] else 2)
            except Exception as e:
                print(name, repr(e), flush=True)
                os._exit(1)
        print(name, os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]), flush=True)
"""


def test_every_entry_point_may_be_a_process_first_call():
    """What the entry points need of torch is looked up by whichever is called first."""
    out = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, cwd=ROOT,
                         env={**os.environ, "PYTHONPATH": f"{ROOT}:{ROOT}/tests"}, check=True).stdout
    assert len(out.splitlines()) == 11 and all(line.endswith(" 0") for line in out.splitlines()), out


def test_forward_workspaces_hold_the_copies_that_the_header_names():
    """x of 17 to 64 rows that are no whole granules is copied beside weights whose rows are,
    not beside others, in half precision; never in fp32."""
    def size(N, D, ldx, ldg, dtype):
        d = _block.FeedForwardDesc(N, D, 512, 64, ldx, ldg, 0, 0, 0, dtype, 0, 0, 0)
        return _block.size("feed_forward_fwd_workspace_size", d, 1)
    for dtype in (_lib.F16, _lib.BF16):
        assert size(40, 64, 68, 0, dtype) - size(40, 64, 0, 0, dtype) == 40 * 64 * 2
        assert size(40, 64, 68, 68, dtype) == size(40, 64, 0, 68, dtype)
        assert size(16, 64, 68, 0, dtype) == size(16, 64, 0, 0, dtype)
        assert size(65, 64, 68, 68, dtype) - size(65, 64, 0, 68, dtype) == 33 * 256           # 65 * 128 bytes in whole 256
    assert size(64, 64, 65, 0, _lib.F32) == size(64, 64, 0, 0, _lib.F32)


def test_launches_that_cannot_be_are_refused_before_anything_is_enqueued():
    """Weights' gradients of more tiles than one launch takes: an invalid descriptor, with no
    workspace size, whatever the pointers are; smaller ones are none of that."""
    for dtype in (_lib.F16, _lib.BF16):
        for D, F, O in ((1 << 20, 1 << 18, 64), (64, 1 << 20, 1 << 20), (1 << 20, 1 << 20, 1 << 20)):
            d = _block.FeedForwardDesc(8192, D, F, O, 0, 0, 0, 0, 0, dtype, 0, 0, 0)
            assert _block.size("feed_forward_bwd_workspace_size", d) == 0
            assert _block.lib().feed_forward_bwd(ctypes.byref(d), *[4096] * 11, None) == 1
    for dtype in (_lib.F32, _lib.F16, _lib.BF16):
        d = _block.FeedForwardDesc(8192, 1 << 18, 1 << 18, 1 << 18, 0, 0, 0, 0, 0, dtype, 0, 0, 0)
        assert _block.size("feed_forward_bwd_workspace_size", d) > 0


def test_workspaces_of_many_gates_hold_no_records_of_each():
    """Lanes that take whole groups of rows leave one record a workgroup: at most 256 of two
    rows of sums, twice; where a workgroup leaves one for each gate there is one for each."""
    def size(N, C, groups):
        d = _block.ResidualNormDesc(N, C, groups, *[0] * 8, 0, 0, 0, 1, 1e-5, 1.0, 1.0)
        return _block.size("residual_norm_bwd_workspace_size", d)
    for N, C, groups in ((65536, 4096, 65536), (65536, 64, 65536), (4096, 1000, 4096), (3000, 520, 1000)):
        assert size(N, C, groups) <= 513 * 2 * C * 4 + 4096
    assert size(19941, 1001, 69) >= (2 * 256 + 69) * 2 * 1001 * 4
    assert size(8192, 9000, 4096) >= 4096 * 2 * 9000 * 4
    # long groups: whole ones where they keep the lanes at work, which takes more of wide rows
    for N, C, few, many in ((65536, 64, 1024, 2048), (32768, 512, 512, 768), (16384, 1024, 256, 512),
                            (16384, 4096, 128, 192), (16384, 2048, 160, 256), (8192, 8192, 256, 512)):
        assert size(N // few * few, C, few) >= (2 * 256 + few) * 2 * C * 4
        assert size(N // many * many, C, many) <= 513 * 2 * C * 4 + 4096


def test_adamw_refuses_copies_in_a_parameters_memory(monkeypatch):
    """Another tensor's workgroup, or in another type the tensor's own, would read what the copy
    wrote; a copy that is its parameter itself changes nothing."""
    calls = []
    monkeypatch.setattr(_block, "call", lambda *args: calls.append(args))
    head._torch_names()
    monkeypatch.setattr(head, "_current_device", lambda: 1)
    monkeypatch.setattr(head, "_raw_stream", lambda dev: 7)
    state = conv.AdamWState([6, 4, 0], 32, "cpu")
    for name in ("exp_avg", "exp_avg_sq"):
        setattr(state, name, DeviceTensor(*getattr(state, name).shape))
    p, g = ([DeviceTensor(n) for n in state.sizes] for _ in range(2))
    wide = DeviceTensor(4)
    half = DeviceTensor(6, dtype=torch.bfloat16)
    half.data_ptr, wide.data_ptr = p[0].data_ptr, p[0].data_ptr
    conv.adamw(p, g, state, 1, 1.0, copies=[p[0], None, p[2]])
    assert len(calls) == 1
    with pytest.raises(ValueError, match=r"copies\[0\] is in the memory of params\[0\]"):
        conv.adamw(p, g, state, 1, 1.0, copies=[half, None, None])
    with pytest.raises(ValueError, match=r"copies\[1\] is in the memory of params\[0\]"):
        conv.adamw(p, g, state, 1, 1.0, copies=[None, wide, None])
    assert len(calls) == 1
