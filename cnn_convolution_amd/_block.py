"""ctypes view of the block operators' entry points of libim2win_conv2d.so
(declarations in include/im2win_block.h). Argument marshalling only."""
from __future__ import annotations

import ctypes

from . import _lib

# every symbol the header declares
EXPORTS = [
    "feed_forward_saved_size", "feed_forward_fwd_workspace_size", "feed_forward_bwd_workspace_size",
    "feed_forward_fwd", "feed_forward_bwd", "residual_norm_fwd", "residual_norm_bwd_workspace_size",
    "residual_norm_bwd", "adamw_step", "adamw_values",
]

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}
KINDS = {"layer": 0, "rms": 1}
BLOCK = 256                    # elements of an 8-bit state that share a scale

_i64, _i32, _u64, _f64, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_double, ctypes.c_void_p


class FeedForwardDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("N", "D", "F", "O", "ldx", "ldg", "ldu", "ldd", "ldy")] + \
               [(n, _i32) for n in ("dtype", "act", "reserved", "reserved2")]


class ResidualNormDesc(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("N", "C", "groups", "ldb", "ldr", "ldo", "ldy", "lddr", "lddb", "lddo", "lddy")] + \
               [(n, _i32) for n in ("dtype", "branch_dtype", "kind", "post")] + \
               [(n, _f64) for n in ("eps", "residual_scale", "branch_scale")]


class AdamWTensor(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("param", "grad", "copy", "m", "v", "m_scale", "v_scale")] + \
               [("n", _i64), ("first", _i64)] + \
               [(n, _i32) for n in ("param_dtype", "grad_dtype", "copy_dtype", "reserved")] + \
               [("lr", _f64), ("weight_decay", _f64)]


class AdamWDesc(ctypes.Structure):
    _fields_ = [("count", _i64), ("bits", _i32), ("reserved", _i32), ("beta1", _f64), ("beta2", _f64), ("eps", _f64),
                ("grad_scale", _f64), ("seed", _u64), ("step", _i64)]


_bound = None


def lib() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        L = _lib.lib()
        size, status = ctypes.c_size_t, ctypes.c_int
        for name, first, args, res in (
                ("feed_forward_saved_size", [ctypes.POINTER(FeedForwardDesc)], 0, size),
                ("feed_forward_fwd_workspace_size", [ctypes.POINTER(FeedForwardDesc), _i32], 0, size),
                ("feed_forward_bwd_workspace_size", [ctypes.POINTER(FeedForwardDesc)], 0, size),
                ("feed_forward_fwd", [ctypes.POINTER(FeedForwardDesc)], 8, status),
                ("feed_forward_bwd", [ctypes.POINTER(FeedForwardDesc)], 12, status),
                ("residual_norm_fwd", [ctypes.POINTER(ResidualNormDesc)], 11, status),
                ("residual_norm_bwd_workspace_size", [ctypes.POINTER(ResidualNormDesc)], 0, size),
                ("residual_norm_bwd", [ctypes.POINTER(ResidualNormDesc)], 18, status),
                ("adamw_step", [ctypes.POINTER(AdamWDesc), ctypes.POINTER(AdamWTensor)], 4, status),
                ("adamw_values", [_i64], 7, status)):
            f = getattr(L, name)
            f.argtypes = first + [_vp] * args
            f.restype = res
        _bound = L
    return _bound


_functions = {}


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def call(name: str, *args) -> None:
    st = _function(name)(*args)
    if st != 0:
        raise _lib.Conv2dError(st, name)


def size(name: str, *args) -> int:
    return _function(name)(*args)
