"""Binding of the operators around the step (include/zerostep_ops.h): the
functions marshal arguments, libzerostep_ops.so's sm_103a kernels compute.

Matrices are 2-D CUDA tensors whose rows are contiguous (any row stride); the
caller makes the outputs.  8-bit matrices are torch.float8_e4m3fn or
torch.float8_e5m2 tensors with fp32 scales of shape [ceil(cols / 128), rows]
(1x128 blocks) or [ceil(cols / 128), ceil(rows / 128)] (128x128 tiles);
``fp8_empty`` makes a pair whose rows start on 16-byte boundaries, as
``zero_fp8_matmul`` wants them.  Work is enqueued on torch's current stream
unless one is given; a tensor used on another stream than the one it was
allocated on is the caller's to keep alive, as with any torch operator.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from ._abi import ZeroError
from ._ops_abi import (BLOCK, T_BF16, T_E4M3, T_E5M2, T_F16, T_F32, TensorsStat, check, lib)

__all__ = [
    "BLOCK", "TensorList", "TensorsStat", "tensor_list", "new_tensors_stat", "read_tensors_stat",
    "zero_tensors_workspace_bytes", "zero_tensors_norm", "zero_tensors_clip", "fp8_empty",
    "zero_fp8_quantize", "zero_fp8_matmul_workspace_bytes", "zero_fp8_matmul", "read_matmul_error",
    "zero_rmsnorm_fp8", "zero_rmsnorm_workspace_bytes", "zero_rmsnorm_backward",
]

_TYPE = {torch.float16: T_F16, torch.bfloat16: T_BF16, torch.float32: T_F32,
         torch.float8_e4m3fn: T_E4M3, torch.float8_e5m2: T_E5M2}


# The calls below are made once for each layer and product of a step, so the
# marshalling counts: tensors' attributes are read once, and the current device
# and stream come from torch's own bindings without objects around them.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _stream(stream, device: int) -> int:
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _current() -> int:
    """The current device's index (-1 without a device: no tensor matches it)."""
    return _device() if torch.cuda.is_initialized() else -1


def _type(t: torch.Tensor) -> int:
    code = _TYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"no operator takes {t.dtype}")
    return code


def _where(name: str = "") -> None:
    raise ValueError(f"{name or 'tensor'}: CUDA tensor of the current device expected")


def _flat(t: Optional[torch.Tensor], dev: int) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    if t.get_device() != dev or dev < 0:
        _where()
    return t.data_ptr()


def _matrix(t: torch.Tensor, rows: int, cols: int, name: str, dtypes, dev: int) -> Tuple[int, int]:
    """(pointer, row stride) of a [rows, cols] matrix with contiguous rows."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    ld, step = t.stride()
    if rows <= 1:
        # torch gives a single row any stride; no second row is ever reached, so
        # the next multiple of 16 elements serves every alignment rule
        ld = (cols + 15) // 16 * 16
    if step != 1 and cols > 1 or ld < cols:
        raise ValueError(f"{name}: contiguous rows expected, strides {t.stride()}")
    if t.get_device() != dev or dev < 0:
        _where(name)
    return t.data_ptr(), ld


_NONE = (None, 0)


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


_F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
_HALF = (torch.float16, torch.bfloat16)
_FLOAT = (torch.float16, torch.bfloat16, torch.float32)
_F32 = (torch.float32,)


# ----------------------------------------------------------------- many tensors

class TensorList:
    """The pointers, sizes and types of a list of contiguous CUDA tensors, in
    the form the library reads; keeps the tensors alive.  A program whose
    gradients stay where they are makes it once."""

    def __init__(self, tensors: Sequence[torch.Tensor]):
        self.tensors = list(tensors)
        n = self.n = len(self.tensors)
        dev = self.device = _current()
        self.ptr = (ctypes.c_void_p * max(n, 1))(*[_flat(t, dev) for t in self.tensors])
        self.numel = (ctypes.c_int64 * max(n, 1))(*[t.numel() for t in self.tensors])
        self.type = (ctypes.c_int32 * max(n, 1))(*[_type(t) for t in self.tensors])


Tensors = Union[TensorList, Sequence[torch.Tensor]]


def tensor_list(tensors: Tensors) -> TensorList:
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def new_tensors_stat(device="cuda") -> torch.Tensor:
    """A device-resident zero_tensors_stat (16 bytes: sumsq, norm, found_inf)."""
    return torch.zeros(ctypes.sizeof(TensorsStat), dtype=torch.uint8, device=device)


def read_tensors_stat(stat: torch.Tensor) -> TensorsStat:
    """Copy a device stat to the host (synchronises with its stream)."""
    return TensorsStat.from_buffer_copy(bytes(stat.cpu().numpy().tobytes()))


def zero_tensors_workspace_bytes(tensors: Tensors) -> int:
    """Workspace bytes of zero_tensors_norm (zero-fill it before first use)."""
    l = tensor_list(tensors)
    n = lib().zero_tensors_workspace_bytes(l.n, l.numel)
    if n == 0:
        raise ZeroError("zero_tensors_workspace_bytes", -1)
    return n


def zero_tensors_norm(tensors: Tensors, inv_scale: float, stat: torch.Tensor, ws: torch.Tensor,
                      tensor_sumsq: Optional[torch.Tensor] = None, stream=None) -> None:
    """The global norm of the tensors times inv_scale into ``stat``;
    ``tensor_sumsq``: one float64 per tensor, each tensor's sum of squares."""
    l, dev = tensor_list(tensors), _current()
    if l.device != dev:
        _where("tensors")
    if stat.nbytes < 16:
        raise ValueError("stat: 16 bytes expected (new_tensors_stat)")
    if tensor_sumsq is not None and (tensor_sumsq.dtype != torch.float64
                                     or tensor_sumsq.numel() != l.n):
        raise ValueError("tensor_sumsq: one float64 for each tensor expected")
    check("zero_tensors_norm",
          lib().zero_tensors_norm(l.n, l.ptr, l.numel, l.type, inv_scale,
                                  _flat(tensor_sumsq, dev), _flat(stat, dev), _flat(ws, dev),
                                  ws.nbytes, _stream(stream, dev)))


def zero_tensors_clip(tensors: Tensors, out: Optional[Tensors], inv_scale: float, max_norm: float,
                      stat: torch.Tensor, stream=None) -> None:
    """out = tensors * inv_scale * min(1, max_norm / (norm + 1e-6)), in place
    with ``out`` None; max_norm 0 does not clip.  Under a loss scale S the norm's
    inv_scale is 1 / S; into the step's flat buffer it is 1 here, for the step
    divides by S itself."""
    l, dev = tensor_list(tensors), _current()
    o = tensor_list(out) if out is not None else None
    if l.device != dev or o is not None and o.device != dev:
        _where("tensors")
    if o is not None and (o.n != l.n or bytes(o.numel) != bytes(l.numel)):
        raise ValueError("out: as many tensors of the same sizes expected")
    if stat.nbytes < 16:
        raise ValueError("stat: 16 bytes expected (new_tensors_stat)")
    check("zero_tensors_clip",
          lib().zero_tensors_clip(l.n, l.ptr, l.numel, l.type, o.ptr if o is not None else None,
                                  o.type if o is not None else None, inv_scale, max_norm,
                                  _flat(stat, dev), _stream(stream, dev)))


# ----------------------------------------------------------------- 8-bit matrices

def fp8_empty(rows: int, cols: int, dtype: torch.dtype = torch.float8_e4m3fn, tile: bool = False,
              device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """(values, scales) of an 8-bit matrix, uninitialised, rows on 16-byte boundaries."""
    pitch = (cols + 15) // 16 * 16
    q = torch.empty(rows, pitch, dtype=dtype, device=device)[:, :cols]
    s = torch.empty(_blocks(cols), _blocks(rows) if tile else rows, dtype=torch.float32,
                    device=device)
    return q, s


def zero_fp8_quantize(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                      s: Optional[torch.Tensor] = None, qt: Optional[torch.Tensor] = None,
                      st: Optional[torch.Tensor] = None, tile: bool = False, stream=None) -> None:
    """x in 8 bits with a scale for each 1x128 block (or 128x128 tile) into
    (q, s), and its transpose, blocks along x's rows, into (qt, st)."""
    if x.dim() != 2:
        raise ValueError("x: matrix expected")
    (rows, cols), dev = x.shape, _current()
    px, ldx = _matrix(x, rows, cols, "x", _FLOAT, dev)
    if (q is None) != (s is None) or (qt is None) != (st is None) or (q is None and qt is None):
        raise ValueError("(q, s), (qt, st) or both expected")
    if q is not None and qt is not None and q.dtype != qt.dtype:
        raise TypeError("q and qt: one 8-bit type expected")
    kb, rb = _blocks(cols), _blocks(rows)
    pq, ldq = _matrix(q, rows, cols, "q", _F8, dev) if q is not None else _NONE
    ps, lds = _matrix(s, kb, rb if tile else rows, "s", _F32, dev) if q is not None else _NONE
    pqt, ldqt = _matrix(qt, cols, rows, "qt", _F8, dev) if qt is not None else _NONE
    pst, ldst = _matrix(st, rb, kb if tile else cols, "st", _F32, dev) if qt is not None else _NONE
    check("zero_fp8_quantize",
          lib().zero_fp8_quantize(px, _TYPE[x.dtype], rows, cols, ldx,
                                  _TYPE[(q if q is not None else qt).dtype], tile, pq, ldq, ps, lds,
                                  pqt, ldqt, pst, ldst, _stream(stream, dev)))


def zero_fp8_matmul_workspace_bytes(m: int, n: int, k: int) -> int:
    """Workspace bytes of zero_fp8_matmul (zero-fill it before first use)."""
    b = lib().zero_fp8_matmul_workspace_bytes(m, n, k)
    if b == 0:
        raise ZeroError("zero_fp8_matmul_workspace_bytes", -1)
    return b


def zero_fp8_matmul(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                    out: torch.Tensor, ws: torch.Tensor, add: bool = False, stream=None) -> None:
    """out[m, n] (+)= a[m, k] b[n, k]^T with a's scales for 1x128 blocks and
    b's, by their shape, for 128x128 tiles or 1x128 blocks."""
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a, b: matrices expected")
    (m, k), n, dev = a.shape, b.shape[0], _current()
    pa, lda = _matrix(a, m, k, "a", _F8, dev)
    pb, ldb = _matrix(b, n, k, "b", _F8, dev)
    kb = _blocks(k)
    psa, ldsa = _matrix(sa, kb, m, "sa", _F32, dev)
    tile = sb.dim() == 2 and sb.shape[1] != n
    psb, ldsb = _matrix(sb, kb, _blocks(n) if tile else n, "sb", _F32, dev)
    po, ldo = _matrix(out, m, n, "out", _FLOAT, dev)
    check("zero_fp8_matmul",
          lib().zero_fp8_matmul(pa, _TYPE[a.dtype], lda, psa, ldsa, pb, _TYPE[b.dtype], ldb, psb, ldsb,
                                tile, po, _TYPE[out.dtype], ldo, m, n, k, add, _flat(ws, dev),
                                ws.nbytes, _stream(stream, dev)))


def read_matmul_error(ws: torch.Tensor) -> bool:
    """Whether a product with this workspace gave up waiting (synchronises with
    its stream; never expected).  Its output is then undefined, and the
    answer stays until the caller clears the word: ``ws[:4].zero_()``."""
    if not ws.is_contiguous() or ws.nbytes < 4:
        raise ValueError("ws: the product's workspace expected")
    return bool(ws.reshape(-1).view(torch.uint8)[:4].any())


# ----------------------------------------------------------------- root-mean-square norm

def zero_rmsnorm_fp8(x: torch.Tensor, w: torch.Tensor, eps: float,
                     rstd: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                     h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                     q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * w in
    x's type and, in 8 bits with a scale for each 1x128 block, into (q, s)."""
    if x.dim() != 2:
        raise ValueError("x: matrix expected")
    (rows, cols), dev = x.shape, _current()
    if w.numel() != cols or rstd is not None and (rstd.numel() != rows
                                                  or rstd.dtype != torch.float32):
        raise ValueError("w: one element for each column, rstd: one fp32 for each row expected")
    if (q is None) != (s is None):
        raise ValueError("q and s: both or neither expected")
    dt = (x.dtype,)
    px, ldx = _matrix(x, rows, cols, "x", _HALF, dev)
    pr, ldr = _matrix(residual, rows, cols, "residual", dt, dev) if residual is not None else _NONE
    ph, ldh = _matrix(h, rows, cols, "h", dt, dev) if h is not None else _NONE
    py, ldy = _matrix(y, rows, cols, "y", dt, dev) if y is not None else _NONE
    pq, ldq = _matrix(q, rows, cols, "q", _F8, dev) if q is not None else _NONE
    ps, lds = _matrix(s, _blocks(cols), rows, "s", _F32, dev) if q is not None else _NONE
    check("zero_rmsnorm_fp8",
          lib().zero_rmsnorm_fp8(px, ldx, pr, ldr, _flat(w, dev), _type(w), _TYPE[x.dtype], rows, cols,
                                 eps, ph, ldh, py, ldy, _TYPE[q.dtype] if q is not None else T_E4M3,
                                 pq, ldq, ps, lds, _flat(rstd, dev), _stream(stream, dev)))


def zero_rmsnorm_workspace_bytes(rows: int, cols: int) -> int:
    """Workspace bytes of zero_rmsnorm_backward."""
    b = lib().zero_rmsnorm_workspace_bytes(rows, cols)
    if b == 0:
        raise ZeroError("zero_rmsnorm_workspace_bytes", -1)
    return b


def zero_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor,
                          dx: torch.Tensor, dw: Optional[torch.Tensor], ws: Optional[torch.Tensor],
                          dres: Optional[torch.Tensor] = None, add_dw: bool = False,
                          stream=None) -> None:
    """dx (the gradient of x and of the residual) and dw of zero_rmsnorm_fp8,
    with the gradient ``dres`` that reaches h by the residual path added."""
    if dy.dim() != 2:
        raise ValueError("dy: matrix expected")
    (rows, cols), dev = dy.shape, _current()
    if w.numel() != cols or dw is not None and dw.numel() != cols:
        raise ValueError("w, dw: one element for each column expected")
    if rstd.numel() != rows or rstd.dtype != torch.float32:
        raise ValueError("rstd: one fp32 for each row expected")
    if dw is not None and ws is None:
        raise ValueError("ws: a workspace expected (zero_rmsnorm_workspace_bytes)")
    dt = (dy.dtype,)
    pdy, lddy = _matrix(dy, rows, cols, "dy", _HALF, dev)
    ph, ldh = _matrix(h, rows, cols, "h", dt, dev)
    pdr, lddr = _matrix(dres, rows, cols, "dres", dt, dev) if dres is not None else _NONE
    pdx, lddx = _matrix(dx, rows, cols, "dx", dt, dev)
    check("zero_rmsnorm_backward",
          lib().zero_rmsnorm_backward(pdy, lddy, ph, ldh, _flat(w, dev), _type(w), _flat(rstd, dev), pdr,
                                      lddr, _TYPE[dy.dtype], rows, cols, pdx, lddx, _flat(dw, dev),
                                      _type(dw) if dw is not None else T_F32, add_dw, _flat(ws, dev),
                                      ws.nbytes if ws is not None else 0, _stream(stream, dev)))
