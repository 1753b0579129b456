"""ctypes view of the training-head entry points of libim2win_conv2d.so
(declarations in include/im2win_head.h). Argument marshalling only."""
from __future__ import annotations

import ctypes

from . import _lib

# every symbol the header declares
EXPORTS = [
    "dropout_fwd", "layer_norm_fwd", "layer_norm_bwd_workspace_size", "layer_norm_bwd",
    "linear_xent_fwd_workspace_size", "linear_xent_bwd_workspace_size", "linear_xent_fwd", "linear_xent_bwd",
]

_i64, _i32, _u64, _f64 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_double


class DropoutDesc(ctypes.Structure):
    _fields_ = [("n", _i64), ("dtype", _i32), ("reserved", _i32), ("p", _f64), ("seed", _u64), ("offset", _u64)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("N", "C", "P", "ldx", "ldy", "lddx")] + \
               [(n, _i32) for n in ("dtype", "y_dtype", "layout", "reserved")] + \
               [("eps", _f64), ("dropout_p", _f64), ("seed", _u64), ("offset", _u64)]


class LinearXentDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("N", "V", "D", "ldx", "ldw")] + [("dtype", _i32), ("reserved", _i32)]


_bound = None


def lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        L = _lib.lib()
        vp, size = ctypes.c_void_p, ctypes.c_size_t
        for name, desc, args, res in (
                ("dropout_fwd", DropoutDesc, 3, ctypes.c_int),
                ("layer_norm_fwd", LayerNormDesc, 7, ctypes.c_int),
                ("layer_norm_bwd_workspace_size", LayerNormDesc, 0, size),
                ("layer_norm_bwd", LayerNormDesc, 10, ctypes.c_int),
                ("linear_xent_fwd_workspace_size", LinearXentDesc, 0, size),
                ("linear_xent_bwd_workspace_size", LinearXentDesc, 0, size),
                ("linear_xent_fwd", LinearXentDesc, 7, ctypes.c_int),
                ("linear_xent_bwd", LinearXentDesc, 9, ctypes.c_int)):
            f = getattr(L, name)
            f.argtypes = [ctypes.POINTER(desc)] + [vp] * args
            f.restype = res
        _bound = L
    return _bound


_functions = {}


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def call(name: str, desc, *args) -> None:
    st = _function(name)(desc, *args)
    if st != 0:
        raise _lib.Conv2dError(st, name)


def size(name: str, desc) -> int:
    return _function(name)(desc)
