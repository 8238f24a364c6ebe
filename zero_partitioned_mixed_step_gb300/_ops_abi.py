"""ctypes declarations of libzerostep_ops.so (include/zerostep_ops.h)."""
from __future__ import annotations

import ctypes
import os

from . import _build
from ._abi import ZeroError

T_F16, T_BF16, T_F32, T_E4M3, T_E5M2 = 0, 1, 4, 8, 9
BLOCK = 128


class TensorsStat(ctypes.Structure):
    _fields_ = [("sumsq", ctypes.c_double), ("norm", ctypes.c_float),
                ("found_inf", ctypes.c_int32)]


assert ctypes.sizeof(TensorsStat) == 16

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_S = ctypes.c_size_t
SIGNATURES = {
    "zero_tensors_workspace_bytes": ([_I, _P], _S),
    "zero_tensors_norm": ([_I, _P, _P, _P, _F, _P, _P, _P, _S, _P], _I),
    "zero_tensors_clip": ([_I, _P, _P, _P, _P, _P, _F, ctypes.c_double, _P, _P], _I),
    "zero_fp8_quantize": ([_P, _I, _I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P, _I64, _P,
                           _I64, _P], _I),
    "zero_fp8_matmul_workspace_bytes": ([_I64, _I64, _I64], _S),
    "zero_fp8_matmul": ([_P, _I, _I64, _P, _I64, _P, _I, _I64, _P, _I64, _I, _P, _I, _I64, _I64,
                         _I64, _I64, _I, _P, _S, _P], _I),
    "zero_rmsnorm_fp8": ([_P, _I64, _P, _I64, _P, _I, _I, _I64, _I64, _F, _P, _I64, _P, _I64, _I,
                          _P, _I64, _P, _I64, _P, _P], _I),
    "zero_rmsnorm_workspace_bytes": ([_I64, _I64], _S),
    "zero_rmsnorm_backward": ([_P, _I64, _P, _I64, _P, _I, _P, _P, _I64, _I, _I64, _I64, _P, _I64,
                               _P, _I, _I, _P, _S, _P], _I),
}

_lib = None


def lib():
    """Load the in-tree libzerostep_ops.so.  There is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.OPS_LIB):
            raise ImportError(
                "libzerostep_ops.so is not built; run `python -c 'import __graft_entry__ as g; "
                "g.build()'` (nvcc, sm_103a) first")
        so = ctypes.CDLL(_build.OPS_LIB)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(so, name)
            f.argtypes = args
            f.restype = res
        _lib = so
    return _lib


def check(fn: str, code: int) -> None:
    if code:
        raise ZeroError(fn, code)
