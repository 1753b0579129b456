"""Training-head operators on the convolution's features: layer norm over the
channels, dropout, and the softmax cross entropy of a linear classifier, each
with its gradient (definitions in include/im2win_head.h).

    y, mean, rstd = layer_norm(x, weight, bias, layout="nhwc", dropout_p=0.1, seed=step)
    loss, lse = linear_cross_entropy(y, w, target)
    dy, dw = linear_cross_entropy_backward(grad, y, w, target, lse)
    dx, dweight, dbias = layer_norm_backward(dy, x, weight, mean, rstd, dropout_p=0.1, seed=step)

Every operator has an ``_into`` form that takes the caller's outputs and
workspace. All work is enqueued on the current stream of x's device, whichever
device is current; the kernels are in the HIP library, PyTorch provides device
memory and streams.
"""
from __future__ import annotations

from . import _head, _lib
from ._head import DropoutDesc, LayerNormDesc, LinearXentDesc

__all__ = ["dropout", "dropout_into", "layer_norm", "layer_norm_into", "layer_norm_backward",
           "layer_norm_backward_into", "layer_norm_workspace_size", "linear_cross_entropy",
           "linear_cross_entropy_into", "linear_cross_entropy_backward", "linear_cross_entropy_backward_into",
           "linear_cross_entropy_workspace_size"]

_codes = None
_raw_stream = None
_current_device = None


def _torch_names() -> None:
    """What the calls below need of torch, looked up once."""
    global _codes, _raw_stream, _current_device, _F32, _I64
    import torch
    _F32, _I64 = torch.float32, torch.int64
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _codes = {torch.float32: _lib.F32, torch.float16: _lib.F16, torch.bfloat16: _lib.BF16}


def _code(dtype) -> int:
    if _codes is None:
        _torch_names()
    try:
        return _codes[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None


def _device(t, name) -> int:
    """The device index of a device tensor; every call that enqueues begins here."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if _codes is None:
        _torch_names()
    return t.get_device()


def _device_guard(dev):
    import torch
    return torch.cuda.device(dev)


def _enqueue(dev, name, desc, *args) -> None:
    """The library's call on the current stream of device dev. A launch goes to
    the current device, and a device's default stream is the null stream on
    every device: dev has to be the current one."""
    if _current_device() == dev:
        _head.call(name, desc, *args, _raw_stream(dev))
    else:
        with _device_guard(dev):
            _head.call(name, desc, *args, _raw_stream(dev))


def _vector(t, name, n, dev, dtype=None):
    """The pointer of a contiguous vector of n elements, fp32 unless said (None
    stays None)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on the device of x")
    dtype = dtype or _F32
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements")
    return t.data_ptr()


def _contiguous(t, name, shape, dtype, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on the device of x")
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _workspace(ws, need, dev):
    if need == 0:
        return None
    if ws is None:
        raise ValueError(f"a workspace (ws) of {need} bytes is needed")
    if ws.get_device() != dev:
        raise ValueError("ws must be a device tensor on the device of x")
    if not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
        raise ValueError(f"ws must be contiguous with at least {need} bytes")
    return ws.data_ptr()


def _bytes(n, like):
    import torch
    return torch.empty(max(n, 1), dtype=torch.uint8, device=like.device)


# ---- dropout ---------------------------------------------------------------

def dropout_into(x, y, p: float, seed: int, offset: int = 0) -> None:
    """y = dropout(x), both contiguous (y may be x)."""
    dev = _device(x, "x")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    d = DropoutDesc(x.numel(), _code(x.dtype), 0, p, seed, offset)
    out = _contiguous(y, "y", x.shape, x.dtype, dev)
    _enqueue(dev, "dropout_fwd", d, x.data_ptr(), out)


def dropout(x, p: float, seed: int, offset: int = 0):
    """Elements of x dropped with probability p (rounded to 1/65536), the others
    scaled; the same call on dy is the gradient. The generator's blocks number
    offset .. offset + ceil(numel/8) - 1 are used."""
    import torch
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    dropout_into(x, y, p, seed, offset)
    return y


# ---- layer norm --------------------------------------------------------------

def _rows(t, name):
    """(rows, C, row stride) of a tensor [..., C] whose leading dimensions
    collapse into rows of one stride."""
    if t.dim() < 1:
        raise ValueError(f"{name} must have a channel dimension")
    C = t.shape[-1]
    if t.numel() == 0 or t.is_contiguous():
        return (t.numel() // C if C else 0), C, C
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    rows, ld = 1, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != ld * rows:
            raise ValueError(f"{name}: the rows must have one stride")
        rows *= size
    ld = C if ld is None else ld
    if ld < C:
        raise ValueError(f"{name}: rows overlap")
    return rows, C, ld


def _norm_desc(x, layout, y_dtype, eps, dropout_p, seed, offset):
    """(descriptor, number of positions)"""
    lay = _lib.NCHW if layout == "nchw" else _lib.NHWC if layout == "nhwc" else layout
    if lay not in (_lib.NCHW, _lib.NHWC):
        raise ValueError(f"unknown layout {layout!r}")
    if lay == _lib.NHWC:
        N, C, ldx = _rows(x, "x")
        P = 1
    else:
        if x.dim() < 3:
            raise ValueError("an nchw x has at least three dimensions")
        if not x.is_contiguous():
            raise ValueError("an nchw x must be contiguous")
        N, C, ldx = x.shape[0], x.shape[1], 0
        P = 1
        for n in x.shape[2:]:
            P *= n
        if P == 0:                                  # maps without positions: nothing to normalise
            N, P = 0, 1
    return LayerNormDesc(N, C, P, ldx, 0, 0, _code(x.dtype), _code(y_dtype), lay, 0, eps, dropout_p, seed,
                         offset), N * P


def _row_stride(d, t, name, shape, dtype, dev):
    """The row stride of y, dy or dx (0 for nchw)."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a device tensor on the device of x")
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    if t.is_contiguous():
        return 0
    if d.layout != _lib.NHWC:
        raise ValueError(f"an nchw {name} must be contiguous")
    return _rows(t, name)[2]


def layer_norm_into(x, weight, bias, y, mean, rstd, eps: float = 1e-5, *, layout="nhwc", dropout_p: float = 0.0,
                    seed: int = 0, offset: int = 0) -> None:
    """Enqueue y, mean, rstd = layer_norm(x); weight, bias may be None, and mean
    and rstd both None when no backward pass follows."""
    dev = _device(x, "x")
    d, n = _norm_desc(x, layout, y.dtype, eps, dropout_p, seed, offset)
    d.ldy = _row_stride(d, y, "y", x.shape, y.dtype, dev)
    C = d.C
    _enqueue(dev, "layer_norm_fwd", d, x.data_ptr(), _vector(weight, "weight", C, dev), _vector(bias, "bias", C, dev),
             y.data_ptr(), _vector(mean, "mean", n, dev), _vector(rstd, "rstd", n, dev))


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, layout="nhwc", out_dtype=None,
               dropout_p: float = 0.0, seed: int = 0, offset: int = 0):
    """Layer norm over the channels of x: the last dimension ("nhwc", rows of one
    stride) or dimension 1 ("nchw", contiguous), then dropout if dropout_p > 0.
    Returns (y, mean, rstd); y is of out_dtype (default x's; others for fp32 x)."""
    import torch
    _device(x, "x")
    odt = x.dtype if out_dtype is None else out_dtype
    d, _ = _norm_desc(x, layout, odt, eps, dropout_p, seed, offset)
    stat = x.shape[:-1] if d.layout == _lib.NHWC else x.shape[:1] + x.shape[2:]
    y = torch.empty(x.shape, dtype=odt, device=x.device)
    mean = torch.empty(stat, dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    layer_norm_into(x, weight, bias, y, mean, rstd, eps, layout=layout, dropout_p=dropout_p, seed=seed,
                    offset=offset)
    return y, mean, rstd


def layer_norm_workspace_size(x, *, layout="nhwc", y_dtype=None, dropout_p: float = 0.0) -> int:
    """Bytes of workspace of layer_norm_backward_into for this x."""
    d, _ = _norm_desc(x, layout, x.dtype if y_dtype is None else y_dtype, 0.0, dropout_p, 0, 0)
    return _head.size("layer_norm_bwd_workspace_size", d)


def layer_norm_backward_into(dy, x, weight, mean, rstd, dx, dweight, dbias, ws, *, layout="nhwc",
                             dropout_p: float = 0.0, seed: int = 0, offset: int = 0) -> None:
    """Enqueue the gradients of layer_norm; dweight and dbias may both be None
    (then ws may be None too)."""
    dev = _device(x, "x")
    d, n = _norm_desc(x, layout, dy.dtype, 0.0, dropout_p, seed, offset)
    d.ldy = _row_stride(d, dy, "dy", x.shape, dy.dtype, dev)
    d.lddx = _row_stride(d, dx, "dx", x.shape, x.dtype, dev)
    C = d.C
    need = _head.size("layer_norm_bwd_workspace_size", d) if dweight is not None else 0
    _enqueue(dev, "layer_norm_bwd", d, dy.data_ptr(), x.data_ptr(), _vector(weight, "weight", C, dev),
             _vector(mean, "mean", n, dev), _vector(rstd, "rstd", n, dev), dx.data_ptr(),
             _vector(dweight, "dweight", C, dev), _vector(dbias, "dbias", C, dev), _workspace(ws, need, dev))


def layer_norm_backward(dy, x, weight, mean, rstd, *, layout="nhwc", dropout_p: float = 0.0, seed: int = 0,
                        offset: int = 0):
    """(dx, dweight, dbias) of layer_norm for the gradient dy of its y, with the
    mean and rstd it returned and its dropout arguments."""
    import torch
    _device(x, "x")
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    C = x.shape[1] if layout in ("nchw", _lib.NCHW) else x.shape[-1]
    dweight = torch.empty(C, dtype=torch.float32, device=x.device)
    dbias = torch.empty_like(dweight)
    ws = _bytes(layer_norm_workspace_size(x, layout=layout, y_dtype=dy.dtype, dropout_p=dropout_p), x)
    layer_norm_backward_into(dy, x, weight, mean, rstd, dx, dweight, dbias, ws, layout=layout, dropout_p=dropout_p,
                             seed=seed, offset=offset)
    return dx, dweight, dbias


# ---- softmax cross entropy of a linear classifier ---------------------------------

def _xent_desc(x, w):
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [N][D] and w [V][D]")
    if x.dtype is not w.dtype:
        raise TypeError("x and w must share a dtype")
    N, D = x.shape
    return LinearXentDesc(N, w.shape[0], D, D if x.is_contiguous() else _rows(x, "x")[2],
                          D if w.is_contiguous() else _rows(w, "w")[2], _code(x.dtype), 0)


def _same_device(x, w) -> int:
    dev = _device(x, "x")
    if w.get_device() != dev:
        raise ValueError("w must be a device tensor on the device of x")
    return dev


def _row_start(t, name, D, ld):
    """The pointer of rows of D elements, ld apart: whole 16-byte granules are read
    in place and start on one, other rows are copied first and start anywhere."""
    p, size = t.data_ptr(), t.element_size()
    if p % 16 and D * size % 16 == 0 and ld * size % 16 == 0:
        raise ValueError(f"{name} must start on a 16-byte boundary, its rows being whole 16-byte pieces "
                         f"(a view that does not can be cloned)")
    return p


def linear_cross_entropy_workspace_size(x, w, *, backward: bool = False) -> int:
    """Bytes of workspace of linear_cross_entropy_into, or with ``backward`` of
    both that and linear_cross_entropy_backward_into."""
    d = _xent_desc(x, w)
    n = _head.size("linear_xent_fwd_workspace_size", d)
    return max(n, _head.size("linear_xent_bwd_workspace_size", d)) if backward else n


def linear_cross_entropy_into(x, w, target, loss, lse, ws) -> None:
    """Enqueue loss, lse = linear_cross_entropy(x, w, target). x and w whose rows and
    row strides are multiples of 16 bytes have to start on a 16-byte boundary."""
    dev = _same_device(x, w)
    d = _xent_desc(x, w)
    N = x.shape[0]
    _enqueue(dev, "linear_xent_fwd", d, _row_start(x, "x", d.D, d.ldx), _row_start(w, "w", d.D, d.ldw),
             _vector(target, "target", N, dev, _I64),
             _vector(loss, "loss", N, dev), _vector(lse, "lse", N, dev),
             _workspace(ws, _head.size("linear_xent_fwd_workspace_size", d), dev))


def linear_cross_entropy(x, w, target):
    """Softmax cross entropy of the logits x w^T (never stored) with int64
    targets: per-row (loss, lse) in fp32. Rows whose target is outside [0, V)
    are masked: both are 0. x and w whose rows and row strides are multiples of
    16 bytes have to start on a 16-byte boundary."""
    import torch
    loss = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    linear_cross_entropy_into(x, w, target, loss, lse, _bytes(linear_cross_entropy_workspace_size(x, w), x))
    return loss, lse


def linear_cross_entropy_backward_into(grad, x, w, target, lse, dx, dw, ws) -> None:
    """Enqueue the gradients of linear_cross_entropy for the per-row gradient
    grad (fp32 [N]) of its loss. w as in linear_cross_entropy_into; x may start
    anywhere."""
    dev = _same_device(x, w)
    d = _xent_desc(x, w)
    N = x.shape[0]
    _enqueue(dev, "linear_xent_bwd", d, _vector(grad, "grad", N, dev), x.data_ptr(),
             _row_start(w, "w", d.D, d.ldw), _vector(target, "target", N, dev, _I64), _vector(lse, "lse", N, dev),
             _contiguous(dx, "dx", x.shape, x.dtype, dev), _contiguous(dw, "dw", w.shape, w.dtype, dev),
             _workspace(ws, _head.size("linear_xent_bwd_workspace_size", d), dev))


def linear_cross_entropy_backward(grad, x, w, target, lse):
    """(dx, dw) of linear_cross_entropy for the per-row gradient grad of its loss."""
    import torch
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty(w.shape, dtype=w.dtype, device=x.device)
    n = _head.size("linear_xent_bwd_workspace_size", _xent_desc(x, w))
    linear_cross_entropy_backward_into(grad, x, w, target, lse, dx, dw, _bytes(n, x))
    return dx, dw
