"""Block operators of a training head: a gated feed-forward block, the norms before
and after a block fused with its gate and residual scale, each with its gradient,
and an AdamW step over many tensors with states in 32 or in 8 bits (definitions in
include/im2win_block.h).

    y, saved = feed_forward(x, w_gate, w_up, w_down)
    out, h, stats = residual_norm(y, residual, gate=gate, post_weight=pw, weight=w)
    dresidual, dy, grads = residual_norm_backward(dh, dout, y, out, stats, gate=gate, post_weight=pw, weight=w)
    dx, dw_gate, dw_up, dw_down = feed_forward_backward(dy, x, w_gate, w_up, w_down, saved)
    adamw(params, grads, state, step, lr)

Every operator has an ``_into`` form that takes the caller's outputs and workspace
(adamw updates in place). All work is enqueued on the current stream of x's device,
whichever device is current; the kernels are in the HIP library, PyTorch provides
device memory and streams.
"""
from __future__ import annotations

import ctypes
from array import array

from . import _block, _lib, head
from ._block import AdamWDesc, AdamWTensor, FeedForwardDesc, ResidualNormDesc
from .head import _bytes, _code, _contiguous, _device, _row_start, _rows, _vector, _workspace

__all__ = ["feed_forward", "feed_forward_into", "feed_forward_backward", "feed_forward_backward_into",
           "feed_forward_workspace_size", "feed_forward_saved_size", "residual_norm", "residual_norm_into",
           "residual_norm_backward", "residual_norm_backward_into", "residual_norm_workspace_size", "AdamWState",
           "adamw", "adamw_state", "adamw_state_values", "adamw_state_values_into"]


def _enqueue(dev, name, *args) -> None:
    """The library's call on the current stream of device dev, with dev the current
    device (a launch goes to that one)."""
    if head._current_device() == dev:
        _block.call(name, *args, head._raw_stream(dev))
    else:
        with head._device_guard(dev):
            _block.call(name, *args, head._raw_stream(dev))


def _stride(t, name, dev, dtype, shape):
    """The row stride of a tensor of this device, type and shape (0: contiguous)."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on the same device as the others")
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    return 0 if t.is_contiguous() else _rows(t, name)[2]


# ---- gated feed-forward block ----------------------------------------------------

def _ff_desc(x, w_gate, w_up, w_down, y, activation):
    """(descriptor, device); y: y or dy, or None where its strides do not count."""
    dev = _device(x, "x")
    dtype = x.dtype
    N, D, ldx = _rows(x, "x")
    shape_g, shape_d = w_gate.shape, w_down.shape
    if len(shape_g) != 2 or len(shape_d) != 2 or shape_g[1] != D or shape_d[1] != shape_g[0]:
        raise ValueError("x must be [..., D], w_gate and w_up [F][D], w_down [O][F]")
    F, O = shape_g[0], shape_d[0]
    try:
        act = _block.ACTIVATIONS[activation]
    except KeyError:
        raise ValueError(f"unknown activation {activation!r}") from None
    return FeedForwardDesc(N, D, F, O, ldx, _stride(w_gate, "w_gate", dev, dtype, shape_g) or D,
                           _stride(w_up, "w_up", dev, dtype, shape_g) or D,
                           _stride(w_down, "w_down", dev, dtype, shape_d) or F,
                           0 if y is None else _stride(y, "y and dy", dev, dtype, x.shape[:-1] + (O,)) or O,
                           _code(dtype), act, 0, 0), dev


def _ff_inputs(d, x, w_gate, w_up, w_down):
    return (_row_start(x, "x", d.D, d.ldx), _row_start(w_gate, "w_gate", d.D, d.ldg),
            _row_start(w_up, "w_up", d.D, d.ldu), _row_start(w_down, "w_down", d.F, d.ldd))


def _saved(saved, d, dev):
    need = _block.size("feed_forward_saved_size", d)
    if saved.get_device() != dev or not saved.is_contiguous() or saved.numel() * saved.element_size() < need:
        raise ValueError(f"saved must be a contiguous device tensor of at least {need} bytes on the device of x")
    return saved.data_ptr()


def feed_forward_saved_size(x, w_gate) -> int:
    """Bytes of ``saved`` for this x and w_gate [F][D]."""
    N, D, _ = _rows(x, "x")
    return _block.size("feed_forward_saved_size", FeedForwardDesc(N, D, w_gate.shape[0], 1, 0, 0, 0, 0, 0,
                                                                  _code(x.dtype), 0, 0, 0))


def feed_forward_workspace_size(x, w_gate, w_up, w_down, *, saved: bool = False, dy=None) -> int:
    """Bytes of workspace of feed_forward_into, with ``saved`` or without, or, with
    ``dy``, of both that and feed_forward_backward_into."""
    d, _ = _ff_desc(x, w_gate, w_up, w_down, dy, "silu")
    n = _block.size("feed_forward_fwd_workspace_size", d, int(saved))
    return n if dy is None else max(n, _block.size("feed_forward_bwd_workspace_size", d))


def feed_forward_into(x, w_gate, w_up, w_down, y, saved, ws, activation: str = "silu") -> None:
    """Enqueue y = feed_forward(x); saved: feed_forward_saved_size bytes for the
    backward pass, or None. x and the weights whose rows and row strides are multiples
    of 16 bytes have to start on a 16-byte boundary."""
    d, dev = _ff_desc(x, w_gate, w_up, w_down, y, activation)
    need = _block.size("feed_forward_fwd_workspace_size", d, int(saved is not None))
    _enqueue(dev, "feed_forward_fwd", d, *_ff_inputs(d, x, w_gate, w_up, w_down), y.data_ptr(),
             None if saved is None else _saved(saved, d, dev), _workspace(ws, need, dev))


def feed_forward(x, w_gate, w_up, w_down, activation: str = "silu", *, save: bool = True):
    """(act(x w_gate^T) * (x w_up^T)) w_down^T over the last dimension of x, all of one
    type: (y, saved), with saved for feed_forward_backward (None without ``save``).
    activation: "silu", "gelu", "gelu_tanh", "relu" or "sigmoid"."""
    import torch
    _device(x, "x")
    y = torch.empty(x.shape[:-1] + (w_down.shape[0],), dtype=x.dtype, device=x.device)
    saved = _bytes(feed_forward_saved_size(x, w_gate), x) if save else None
    ws = _bytes(feed_forward_workspace_size(x, w_gate, w_up, w_down, saved=save), x)
    feed_forward_into(x, w_gate, w_up, w_down, y, saved, ws, activation)
    return y, saved


def feed_forward_backward_into(dy, x, w_gate, w_up, w_down, saved, dx, dw_gate, dw_up, dw_down, ws,
                               activation: str = "silu") -> None:
    """Enqueue the gradients of feed_forward for the gradient dy of its y, with what it
    saved for the same x and weights (its activation and slopes among it: ``activation`` is
    checked and has no other effect). dy is read as x is."""
    d, dev = _ff_desc(x, w_gate, w_up, w_down, dy, activation)
    need = _block.size("feed_forward_bwd_workspace_size", d)
    _enqueue(dev, "feed_forward_bwd", d, _row_start(dy, "dy", d.O, d.ldy), *_ff_inputs(d, x, w_gate, w_up, w_down),
             _saved(saved, d, dev), _contiguous(dx, "dx", x.shape, x.dtype, dev),
             _contiguous(dw_gate, "dw_gate", w_gate.shape, x.dtype, dev),
             _contiguous(dw_up, "dw_up", w_up.shape, x.dtype, dev),
             _contiguous(dw_down, "dw_down", w_down.shape, x.dtype, dev), _workspace(ws, need, dev))


def feed_forward_backward(dy, x, w_gate, w_up, w_down, saved, activation: str = "silu"):
    """(dx, dw_gate, dw_up, dw_down) of feed_forward for the gradient dy of its y, with
    the activation of the forward pass that ``saved`` is from."""
    import torch
    _device(x, "x")
    out = [torch.empty(t.shape, dtype=x.dtype, device=x.device) for t in (x, w_gate, w_up, w_down)]
    d, _ = _ff_desc(x, w_gate, w_up, w_down, dy, activation)
    ws = _bytes(_block.size("feed_forward_bwd_workspace_size", d), x)
    feed_forward_backward_into(dy, x, w_gate, w_up, w_down, saved, *out, ws, activation)
    return tuple(out)


# ---- norms around a residual sum ---------------------------------------------------

def _rn_desc(branch, gate, kind, post, eps, residual_scale, branch_scale, residual_dtype):
    """(descriptor, device, rows); the strides are 0 (contiguous rows)."""
    dev = _device(branch, "branch")
    N, C, ldb = _rows(branch, "branch")
    try:
        k = _block.KINDS[kind]
    except KeyError:
        raise ValueError(f"unknown kind {kind!r}") from None
    groups = 0
    if gate is not None:
        if gate.shape[-1] != C or gate.dim() > 2:
            raise ValueError(f"gate must be [{C}] or [groups][{C}]")
        groups = gate.numel() // C
        if groups < 1 or N % groups:
            raise ValueError(f"the gate's {groups} groups must divide the {N} rows")
    return ResidualNormDesc(N, C, groups, ldb, 0, 0, 0, 0, 0, 0, 0, _code(residual_dtype), _code(branch.dtype), k,
                            int(bool(post)), eps, residual_scale, branch_scale), dev


def _row_tensor(t, name, shape, dtype, dev):
    """(pointer, row stride)"""
    return t.data_ptr(), _stride(t, name, dev, dtype, shape)


def _no_post(post, **vectors):
    if not post:
        for name, t in vectors.items():
            if t is not None:
                raise ValueError(f"{name}: there is no norm after the block (post=False)")


def _gate(gate, d, dev):
    return _vector(gate, "gate", d.groups * d.C, dev)


def residual_norm_workspace_size(branch, *, gate=None, post: bool = True, residual_dtype=None) -> int:
    """Bytes of workspace of residual_norm_backward_into."""
    d, _ = _rn_desc(branch, gate, "layer", post, 0.0, 1.0, 1.0, residual_dtype or branch.dtype)
    return _block.size("residual_norm_bwd_workspace_size", d)


def residual_norm_into(branch, residual, out, y, stats, eps: float = 1e-5, *, gate=None, post_weight=None,
                       post_bias=None, weight=None, bias=None, kind: str = "layer", post: bool = True,
                       residual_scale: float = 1.0, branch_scale: float = 1.0) -> None:
    """Enqueue out, y, stats = residual_norm(branch, residual); stats may be None
    when no backward pass follows. No tensor may overlap another."""
    d, dev = _rn_desc(branch, gate, kind, post, eps, residual_scale, branch_scale, residual.dtype)
    _no_post(post, post_weight=post_weight, post_bias=post_bias)
    r, d.ldr = _row_tensor(residual, "residual", branch.shape, residual.dtype, dev)
    o, d.ldo = _row_tensor(out, "out", branch.shape, residual.dtype, dev)
    yp, d.ldy = _row_tensor(y, "y", branch.shape, branch.dtype, dev)
    C = d.C
    _enqueue(dev, "residual_norm_fwd", d, branch.data_ptr(), r, _gate(gate, d, dev),
             _vector(post_weight, "post_weight", C, dev), _vector(post_bias, "post_bias", C, dev),
             _vector(weight, "weight", C, dev), _vector(bias, "bias", C, dev), o, yp,
             _vector(stats, "stats", d.N * 4, dev))


def residual_norm(branch, residual, eps: float = 1e-5, *, gate=None, post_weight=None, post_bias=None, weight=None,
                  bias=None, kind: str = "layer", post: bool = True, residual_scale: float = 1.0,
                  branch_scale: float = 1.0):
    """out = residual_scale * residual + branch_scale * gate * (norm(branch) * post_weight
    + post_bias) and y = norm(out) * weight + bias over rows of channels (the last
    dimension, rows of one stride): (out, y, stats). kind: "layer" or "rms", of both
    norms; post=False leaves the first one out. gate: fp32 [C], or [groups][C] with one
    gate for each of as many equal runs of rows (the images of a batch). out is of
    residual's type, y of branch's, which may be a half precision one beside an fp32
    residual; weights and biases are fp32 [C]. stats [rows][4] are for the backward pass."""
    import torch
    _device(branch, "branch")
    out = torch.empty(branch.shape, dtype=residual.dtype, device=branch.device)
    y = torch.empty(branch.shape, dtype=branch.dtype, device=branch.device)
    stats = torch.empty(branch.shape[:-1] + (4,), dtype=torch.float32, device=branch.device)
    residual_norm_into(branch, residual, out, y, stats, eps, gate=gate, post_weight=post_weight, post_bias=post_bias,
                       weight=weight, bias=bias, kind=kind, post=post, residual_scale=residual_scale,
                       branch_scale=branch_scale)
    return out, y, stats


def residual_norm_backward_into(dy, dout, branch, out, stats, dresidual, dbranch, ws, *, gate=None, post_weight=None,
                                post_bias=None, weight=None, dgate=None, dpost_weight=None, dpost_bias=None,
                                dweight=None, dbias=None, kind: str = "layer", post: bool = True,
                                residual_scale: float = 1.0, branch_scale: float = 1.0) -> None:
    """Enqueue the gradients of residual_norm for the gradients dy of its y and dout of
    its out (None: 0). Each of the parameters' gradients may be None, and ws too if
    all are."""
    d, dev = _rn_desc(branch, gate, kind, post, 0.0, residual_scale, branch_scale, out.dtype)
    _no_post(post, post_weight=post_weight, post_bias=post_bias, dpost_weight=dpost_weight, dpost_bias=dpost_bias)
    if dgate is not None and gate is None:
        raise ValueError("dgate: there is no gate")
    o, d.ldo = _row_tensor(out, "out", branch.shape, out.dtype, dev)
    gy, d.lddy = _row_tensor(dy, "dy", branch.shape, branch.dtype, dev)
    go = None
    if dout is not None:
        go, d.lddo = _row_tensor(dout, "dout", branch.shape, out.dtype, dev)
    dr, d.lddr = _row_tensor(dresidual, "dresidual", branch.shape, out.dtype, dev)
    db, d.lddb = _row_tensor(dbranch, "dbranch", branch.shape, branch.dtype, dev)
    C = d.C
    sums = any(t is not None for t in (dgate, dpost_weight, dpost_bias, dweight, dbias))
    need = _block.size("residual_norm_bwd_workspace_size", d) if sums else 0
    _enqueue(dev, "residual_norm_bwd", d, gy, go, branch.data_ptr(), o, _vector(stats, "stats", d.N * 4, dev),
             _gate(gate, d, dev), _vector(post_weight, "post_weight", C, dev), _vector(post_bias, "post_bias", C, dev),
             _vector(weight, "weight", C, dev), dr, db, _vector(dgate, "dgate", d.groups * C, dev),
             _vector(dpost_weight, "dpost_weight", C, dev), _vector(dpost_bias, "dpost_bias", C, dev),
             _vector(dweight, "dweight", C, dev), _vector(dbias, "dbias", C, dev), _workspace(ws, need, dev))


def residual_norm_backward(dy, dout, branch, out, stats, *, gate=None, post_weight=None, post_bias=None, weight=None,
                           kind: str = "layer", post: bool = True, residual_scale: float = 1.0,
                           branch_scale: float = 1.0):
    """(dresidual, dbranch, grads) of residual_norm, with its out and stats and its
    arguments; grads is a dict of the parameters' gradients: "weight", "bias", with a
    norm after the block "post_weight" and "post_bias", with a gate "gate"."""
    import torch
    _device(branch, "branch")
    C = branch.shape[-1]
    dr = torch.empty(branch.shape, dtype=out.dtype, device=branch.device)
    db = torch.empty(branch.shape, dtype=branch.dtype, device=branch.device)
    names = ["weight", "bias"] + (["post_weight", "post_bias"] if post else [])
    grads = {n: torch.empty(C, dtype=torch.float32, device=branch.device) for n in names}
    if gate is not None:
        grads["gate"] = torch.empty_like(gate, memory_format=torch.contiguous_format)
    ws = _bytes(residual_norm_workspace_size(branch, gate=gate, post=post, residual_dtype=out.dtype), branch)
    residual_norm_backward_into(dy, dout, branch, out, stats, dr, db, ws, gate=gate, post_weight=post_weight,
                                post_bias=post_bias, weight=weight, kind=kind, post=post,
                                residual_scale=residual_scale, branch_scale=branch_scale,
                                **{"d" + n: g for n, g in grads.items()})
    return dr, db, grads


# ---- AdamW over many tensors ---------------------------------------------------------

# adamw's table of tensors is filled column by column: words of 8 bytes of an AdamWTensor
# (a call with 150 tensors spends its time here: 250 us field by field, 140 so)
_TABLE_WORDS = ctypes.sizeof(AdamWTensor) // 8


def _data_ptr(t):
    return t.data_ptr()


class AdamWState:
    """The states of ``adamw`` for a list of tensors, in one buffer each: tensor i's
    elements are at first[i] .. first[i] + sizes[i], every tensor starting at a multiple
    of 256 (what lies between is 0).

    bits 32: exp_avg, exp_avg_sq fp32. bits 8: int8 and uint8 codes, with the scales
    exp_avg_scale, exp_avg_sq_scale (fp32, one per 256 elements). The buffers may be
    saved and copied back; adamw_state_values gives what they stand for."""

    def __init__(self, sizes, bits, device):
        import torch
        if bits not in (32, 8):
            raise ValueError("bits must be 32 or 8")
        self.bits, self.sizes, self.first, n = bits, list(sizes), [], 0
        for k in self.sizes:
            self.first.append(n)
            n += -(-k // _block.BLOCK) * _block.BLOCK
        self.exp_avg = torch.zeros(n, dtype=torch.int8 if bits == 8 else torch.float32, device=device)
        self.exp_avg_sq = torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32, device=device)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if bits == 8:
            self.exp_avg_scale = torch.zeros(n // _block.BLOCK, device=device)
            self.exp_avg_sq_scale = torch.zeros(n // _block.BLOCK, device=device)
        self._numel, self._table = n, (None, None)

    def _entries(self, m, v, ms, vs):
        """The table of tensors with what the state's buffers at these addresses give."""
        if self._table[0] != (m, v, ms, vs):
            table = bytearray(len(self.sizes) * _TABLE_WORDS * 8)
            whole, es = memoryview(table).cast("q"), 1 if self.bits == 8 else 4
            whole[3::_TABLE_WORDS] = array("q", [m + at * es for at in self.first])
            whole[4::_TABLE_WORDS] = array("q", [v + at * es for at in self.first])
            if ms is not None:
                whole[5::_TABLE_WORDS] = array("q", [ms + at // _block.BLOCK * 4 for at in self.first])
                whole[6::_TABLE_WORDS] = array("q", [vs + at // _block.BLOCK * 4 for at in self.first])
                whole[8::_TABLE_WORDS] = array("q", self.first)
            whole[7::_TABLE_WORDS] = array("q", self.sizes)
            self._table = (m, v, ms, vs), bytes(table)
        return bytearray(self._table[1])


def adamw_state(params, bits: int = 32) -> AdamWState:
    """Zero states for the tensors ``params``, all on one device."""
    params = list(params)
    if not params:
        raise ValueError("no tensors")
    dev = _device(params[0], "params[0]")
    for i, p in enumerate(params):
        if p.get_device() != dev:
            raise ValueError(f"params[{i}] must be on the device of params[0]")
    return AdamWState([p.numel() for p in params], bits, params[0].device)


def _state_pointers(state, dev):
    """Pointers of the state's buffers, checked: m, v, and with 8 bits the scales."""
    import torch
    n = state._numel
    types = (torch.int8, torch.uint8) if state.bits == 8 else (torch.float32, torch.float32)
    m, v = (_vector(t, name, n, dev, dtype) for t, name, dtype in (
        (state.exp_avg, "exp_avg", types[0]), (state.exp_avg_sq, "exp_avg_sq", types[1])))
    if state.bits != 8:
        return m, v, None, None
    k = n // _block.BLOCK
    return m, v, _vector(state.exp_avg_scale, "exp_avg_scale", k, dev), \
        _vector(state.exp_avg_sq_scale, "exp_avg_sq_scale", k, dev)


def _checked(tensors, name, sizes, dev):
    """The type codes of contiguous tensors of these sizes on device dev."""
    known, codes = head._codes, []
    for t, n in zip(tensors, sizes):
        if t is None:
            raise ValueError(f"{name}[{len(codes)}] is None: leave its tensor out, with a state of its own")
        if t.get_device() != dev:
            raise ValueError(f"{name}[{len(codes)}] must be on the device of params[0]")
        if t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name}[{len(codes)}] must be a contiguous tensor of {n} elements, as its state is")
        code = known.get(t.dtype)
        codes.append(_code(t.dtype) if code is None else code)
    return codes


def _no_twice(pointers, name, numbers, sizes):
    """Refuses a tensor that is in the list twice (two workgroups would update it at once);
    the pointers as a set."""
    some = set(pointers)
    if len(some) == len(pointers):
        return some
    seen = set()
    for i, p in zip(numbers, pointers):
        if sizes[i] and p in seen:
            raise ValueError(f"{name}[{i}] is in the list twice")
        seen.add(p)
    return some


def _no_parameter(copies, params, numbers, codes, types, sizes):
    """Refuses a copy in a parameter's memory, unless it is that parameter itself."""
    at = {p: i for i, p in enumerate(params) if sizes[i]}
    for i, c, code in zip(numbers, copies, codes):
        if sizes[i] and c in at and (at[c] != i or types[i] != code):
            raise ValueError(f"copies[{i}] is in the memory of params[{at[c]}]")


def _each(value, name, count):
    if isinstance(value, (int, float)):
        return [float(value)] * count
    value = [float(v) for v in value]
    if len(value) != count:
        raise ValueError(f"{name} must be a number or one for each of the {count} tensors")
    return value


def adamw(params, grads, state: AdamWState, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
          weight_decay=0.0, *, grad_scale=1.0, copies=None, seed: int = 0, lr_scale=None) -> None:
    """Enqueue one AdamW step: every tensor of ``params`` and ``state`` (adamw_state of
    these tensors) is updated in place from ``grads``, all contiguous and each of any of
    the three types; ``copies``, where given, receive the new parameters in their own
    types (None entries are left out). Parameters, copies and states must not overlap.

    step: the number of this step, from 1 on. lr, weight_decay: numbers, or one for each
    tensor. grad_scale multiplies the gradients (1 / loss scale). seed: of the numbers
    that round 8-bit states. For steps captured into a graph, step may be an int64 device
    tensor of one element, grad_scale an fp32 one, and lr_scale an fp32 one that
    multiplies every lr."""
    params, grads = list(params), list(grads)
    count = len(params)
    if count == 0 or len(grads) != count or len(state.sizes) != count:
        raise ValueError("params, grads and state must be of the same, non-zero number of tensors")
    dev = _device(params[0], "params[0]")
    words, types = _TABLE_WORDS, _checked(params, "params", state.sizes, dev)
    table = state._entries(*_state_pointers(state, dev))
    whole, real = memoryview(table).cast("q"), memoryview(table).cast("d")
    whole[0::words] = pointers = array("q", map(_data_ptr, params))
    held = _no_twice(pointers, "params", range(count), state.sizes)
    whole[9::words] = array("q", [p | g << 32 for p, g in zip(types, _checked(grads, "grads", state.sizes, dev))])
    whole[1::words] = array("q", map(_data_ptr, grads))
    if copies is not None:
        copies = list(copies)
        if len(copies) != count:
            raise ValueError("copies must have an entry for each tensor")
        some = [i for i, c in enumerate(copies) if c is not None]
        codes = _checked([copies[i] for i in some], "copies", [state.sizes[i] for i in some], dev)
        for i, code in zip(some, codes):
            whole[i * words + 2], whole[i * words + 10] = copies[i].data_ptr(), code
        to = [whole[i * words + 2] for i in some]
        if not held.isdisjoint(_no_twice(to, "copies", some, state.sizes)):
            _no_parameter(to, pointers, some, codes, types, state.sizes)
    real[11::words] = array("d", _each(lr, "lr", count))
    real[12::words] = array("d", _each(weight_decay, "weight_decay", count))
    step_ptr = scale_ptr = None
    if not isinstance(step, int):
        step_ptr, step = _vector(step, "step", 1, dev, head._I64), 0
    elif step < 1:
        raise ValueError("steps are numbered from 1 on")
    if not isinstance(grad_scale, (int, float)):
        scale_ptr, grad_scale = _vector(grad_scale, "grad_scale", 1, dev), 1.0
    d = AdamWDesc(count, state.bits, 0, beta1, beta2, eps, grad_scale, seed, step)
    entries = (AdamWTensor * count).from_buffer(table)
    _enqueue(dev, "adamw_step", d, entries, step_ptr, scale_ptr, _vector(lr_scale, "lr_scale", 1, dev))


def adamw_state_values_into(state: AdamWState, exp_avg, exp_avg_sq) -> None:
    """Enqueue what the 8-bit ``state`` stands for into two fp32 buffers of its size."""
    if state.bits != 8:
        raise ValueError("32-bit states are their values")
    n = state.exp_avg.numel()
    dev = _device(state.exp_avg, "the state")
    m, v, ms, vs = _state_pointers(state, dev)
    _enqueue(dev, "adamw_values", n, m, v, ms, vs, _vector(exp_avg, "exp_avg", n, dev),
             _vector(exp_avg_sq, "exp_avg_sq", n, dev))


def adamw_state_values(state: AdamWState):
    """(exp_avg, exp_avg_sq) in fp32 in the layout of the state's buffers."""
    import torch
    if state.bits != 8:
        return state.exp_avg, state.exp_avg_sq
    out = [torch.empty(state.exp_avg.numel(), dtype=torch.float32, device=state.exp_avg.device) for _ in range(2)]
    adamw_state_values_into(state, *out)
    return tuple(out)
