"""ctypes declarations of libzerostep_layer.so (include/zerostep_layer.h)."""
from __future__ import annotations

import ctypes
import os
import struct

from . import _build

GATE_NONE, GATE_ONE, GATE_COLS, GATE_ROWS = 0, 1, 2, 3
ACT_SILU, ACT_GELU = 0, 1


class Fp8Form(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("ld", ctypes.c_int64), ("s", ctypes.c_void_p), ("lds", ctypes.c_int64)]


# An Fp8Form's bytes from its members: a third of what making the structure takes.
pack_form = struct.Struct("PqPq").pack
assert struct.calcsize("PqPq") == ctypes.sizeof(Fp8Form)

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_S = ctypes.c_size_t
_M = [_P, _I64]
_FORM = ctypes.c_void_p  # of an Fp8Form, or its bytes
SIGNATURES = {
    "zero_gated_norms_fp8": ([*_M, *_M, _P, _P, _I, _P, _I, _I, _F, _I, _I64, _I64, _F, *_M, *_M, _I, _FORM, _FORM,
                              _FORM, _P, _P, _P], _I),
    "zero_gated_norms_workspace_bytes": ([_I64, _I64], _S),
    "zero_gated_norms_backward": ([*_M, *_M, *_M, *_M, *_M, *_M, _P, _P, _P, _P, _I, _P, _I, _I, _F, _I, _I64, _I64,
                                   *_M, *_M, _P, _P, _P, _I, _I, _P, _S, _P], _I),
    "zero_activation_fp8": ([*_M, *_M, _I, _I, _I64, _I64, *_M, _I, _FORM, _FORM, _FORM, _P], _I),
    "zero_activation_backward_fp8": ([*_M, *_M, *_M, *_M, *_M, _I, _I, _I64, _I64, *_M, *_M, _I, _FORM, _FORM, _FORM,
                                      _FORM, _FORM, _P], _I),
    "zero_fp8_restore": ([_P, _I, _I64, *_M, _P, _P, _I, _I64, _I64, _P, _I, _I64, _FORM, _P], _I),
}

_lib = None


def lib():
    """Load the in-tree libzerostep_layer.so.  There is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LAYER_LIB):
            raise ImportError(
                "libzerostep_layer.so is not built; run `python -c 'import __graft_entry__ as g; "
                "g.build()'` (nvcc, sm_103a) first")
        so = ctypes.CDLL(_build.LAYER_LIB)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(so, name)
            f.argtypes = args
            f.restype = res
        _lib = so
    return _lib
