"""Binding of what lies between a layer's 8-bit products (include/zerostep_layer.h):
the functions marshal arguments, libzerostep_layer.so's sm_103a kernels compute.

Tensors are as in ``ops``: 2-D CUDA tensors with contiguous rows, made by the
caller.  An 8-bit matrix that a call writes is passed as the pair (values, scales)
that ``fp8_empty`` makes, with a scale for each 1x128 block.  A checkpoint is such
a pair in E4M3, or the half tensor itself.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._abi import ZeroError
from ._layer_abi import (ACT_GELU, ACT_SILU, GATE_COLS, GATE_NONE, GATE_ONE, GATE_ROWS, lib, pack_form)
from ._ops_abi import BLOCK, T_E4M3, T_F32, check
from .ops import (_F32, _F8, _FLOAT, _HALF, _NONE, _TYPE, _blocks, _current, _flat, _matrix, _stream, _type, _where)

__all__ = [
    "zero_gated_norms_fp8", "zero_gated_norms_workspace_bytes", "zero_gated_norms_backward",
    "zero_activation_fp8", "zero_activation_backward_fp8", "zero_fp8_restore",
]

Pair = Tuple[torch.Tensor, torch.Tensor]
_E4M3 = (torch.float8_e4m3fn,)
_ACT = {"silu": ACT_SILU, "gelu": ACT_GELU}


def _form(pair: Optional[Pair], rows: int, cols: int, name: str, dtypes, dev: int) -> Optional[bytes]:
    if pair is None:
        return None
    q, s = pair
    pq, ld = _matrix(q, rows, cols, name, dtypes, dev)
    ps, lds = _matrix(s, (cols + BLOCK - 1) // BLOCK, rows, name, _F32, dev)
    return pack_form(pq or 0, ld, ps or 0, lds)


def _some(t: Optional[torch.Tensor], rows: int, cols: int, name: str, dtypes, dev: int) -> Tuple[Optional[int], int]:
    return _NONE if t is None else _matrix(t, rows, cols, name, dtypes, dev)


def _one_type(*pairs: Optional[Pair]) -> int:
    """The 8-bit type of the pairs that are there (E4M3 without any)."""
    dtype = None
    for p in pairs:
        if p is not None:
            if dtype is not None and p[0].dtype != dtype:
                raise TypeError("8-bit outputs: one type expected")
            dtype = p[0].dtype
    return T_E4M3 if dtype is None else _TYPE.get(dtype, -1)


def _vector(t: Optional[torch.Tensor], n: int, name: str, dev: int, dtype=None) -> Optional[int]:
    if t is None:
        return None
    if t.numel() != n or dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: {n} elements{f' of {dtype}' if dtype else ''} expected")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    if t.get_device() != dev or dev < 0:
        _where(name)
    return t.data_ptr()


def _gate_kind(gate: Optional[torch.Tensor], rows: int, cols: int) -> int:
    """By the gate's own dimensions, so that a number's meaning (and whether its gradient is added) does not
    hang on how many rows a call has: two dimensions are a token's, whatever their sizes."""
    if gate is None:
        return GATE_NONE
    if gate.dim() == 2:
        if gate.shape == (rows, 1):
            return GATE_ROWS
    elif gate.numel() == 1:
        return GATE_ONE
    elif gate.shape == (cols,):
        return GATE_COLS
    raise ValueError(f"gate: shape {tuple(gate.shape)}, expected () or (1,), {(cols,)} or {(rows, 1)}")


def _norm_weights(w_pre, w_post, cols, dev):
    """(w_post, w_pre, their type)."""
    if w_post is not None and w_post.dtype != w_pre.dtype:
        raise TypeError("w_pre, w_post: one type expected")
    return _vector(w_post, cols, "w_post", dev), _vector(w_pre, cols, "w_pre", dev), _type(w_pre)


# ----------------------------------------------------------------- norms around a block

def zero_gated_norms_fp8(o: torch.Tensor, x: torch.Tensor, w_pre: torch.Tensor, eps: float, h: torch.Tensor,
                         w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                         scale: float = 1.0, y: Optional[torch.Tensor] = None, y8: Optional[Pair] = None,
                         o8: Optional[Pair] = None, h8: Optional[Pair] = None,
                         rstd_post: Optional[torch.Tensor] = None, rstd_pre: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """h = scale * x + gate * norm(o) with w_post (or gate * o without), y = norm(h) with
    w_pre, in o's type and, in 8 bits, into y8; checkpoints of o and h into o8 and
    h8.  gate: one number as [] or [1], [cols], or [rows, 1], a number a token."""
    if o.dim() != 2:
        raise ValueError("o: matrix expected")
    (rows, cols), dev = o.shape, _current()
    dt = (o.dtype,)
    po, ldo = _matrix(o, rows, cols, "o", _HALF, dev)
    px, ldx = _matrix(x, rows, cols, "x", dt, dev)
    ph, ldh = _matrix(h, rows, cols, "h", dt, dev)
    py, ldy = _some(y, rows, cols, "y", dt, dev)
    kind = _gate_kind(gate, rows, cols)
    check("zero_gated_norms_fp8",
          lib().zero_gated_norms_fp8(
              po, ldo, px, ldx, *_norm_weights(w_pre, w_post, cols, dev), _flat(gate, dev), kind,
              _type(gate) if kind else T_F32, scale, _TYPE[o.dtype], rows, cols, eps, ph, ldh, py, ldy, _one_type(y8),
              _form(y8, rows, cols, "y8", _F8, dev), _form(o8, rows, cols, "o8", _E4M3, dev),
              _form(h8, rows, cols, "h8", _E4M3, dev),
              _vector(rstd_post, rows, "rstd_post", dev, torch.float32),
              _vector(rstd_pre, rows, "rstd_pre", dev, torch.float32),
              _stream(stream, dev)))


def zero_gated_norms_workspace_bytes(rows: int, cols: int) -> int:
    """Workspace bytes of zero_gated_norms_backward."""
    b = lib().zero_gated_norms_workspace_bytes(rows, cols)
    if b == 0:
        raise ZeroError("zero_gated_norms_workspace_bytes", -1)
    return b


def _kept(t, s, rows, cols, name, dtype, dev):
    """(pointer, stride, scales, their stride) of a checkpoint."""
    if s is None:
        return (*_matrix(t, rows, cols, name, (dtype,), dev), None, 0)
    return (*_matrix(t, rows, cols, name, _E4M3, dev), *_matrix(s, _blocks(cols), rows, name + " scales", _F32, dev))


def zero_gated_norms_backward(dy: torch.Tensor, o: torch.Tensor, h: torch.Tensor, w_pre: torch.Tensor,
                              rstd_pre: torch.Tensor, d_o: torch.Tensor, dx: torch.Tensor,
                              ws: Optional[torch.Tensor], so: Optional[torch.Tensor] = None,
                              sh: Optional[torch.Tensor] = None, dh: Optional[torch.Tensor] = None,
                              w_post: Optional[torch.Tensor] = None, rstd_post: Optional[torch.Tensor] = None,
                              gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                              dw_pre: Optional[torch.Tensor] = None, dw_post: Optional[torch.Tensor] = None,
                              dgate: Optional[torch.Tensor] = None, add: bool = False, stream=None) -> None:
    """The gradients of zero_gated_norms_fp8 from dy and the gradient dh that reaches h
    along the stream: d_o, dx (the stream's), dw_pre, dw_post, dgate.  o, h: what was
    kept, both halves, or both E4M3 with the scales so and sh.  add: dw_pre, dw_post and the dgate of
    one number or of channels are added to what is there; a token's dgate is written."""
    if dy.dim() != 2:
        raise ValueError("dy: matrix expected")
    (rows, cols), dev = dy.shape, _current()
    if (so is None) != (sh is None):
        raise ValueError("so and sh: both or neither expected")
    if w_post is not None and rstd_post is None:
        raise ValueError("rstd_post: needed with w_post")
    if w_post is None and dw_post is not None or gate is None and dgate is not None:
        raise ValueError("a gradient of what is not there")
    dt = dy.dtype
    pdy, lddy = _matrix(dy, rows, cols, "dy", _HALF, dev)
    kind = _gate_kind(gate, rows, cols)
    grad_type = T_F32
    for g in (dw_pre, dw_post, dgate):
        if g is not None:
            grad_type = _type(g)
            if g.dtype != (dw_pre if dw_pre is not None else dw_post if dw_post is not None else dgate).dtype:
                raise TypeError("dw_pre, dw_post, dgate: one type expected")
    if ws is None and (dw_pre is not None or dw_post is not None or dgate is not None and kind != GATE_ROWS):
        raise ValueError("ws: a workspace expected (zero_gated_norms_workspace_bytes)")
    check("zero_gated_norms_backward",
          lib().zero_gated_norms_backward(
              pdy, lddy, *_some(dh, rows, cols, "dh", (dt,), dev), *_kept(o, so, rows, cols, "o", dt, dev),
              *_kept(h, sh, rows, cols, "h", dt, dev),
              _vector(rstd_post, rows, "rstd_post", dev, torch.float32),
              _vector(rstd_pre, rows, "rstd_pre", dev, torch.float32), *_norm_weights(w_pre, w_post, cols, dev),
              _flat(gate, dev), kind, _type(gate) if kind else T_F32, scale, _TYPE[dt], rows, cols,
              *_matrix(d_o, rows, cols, "d_o", (dt,), dev), *_matrix(dx, rows, cols, "dx", (dt,), dev),
              _vector(dw_post, cols, "dw_post", dev), _vector(dw_pre, cols, "dw_pre", dev),
              _vector(dgate, 0 if gate is None else gate.numel(), "dgate", dev), grad_type, add, _flat(ws, dev), 0 if ws is None else ws.nbytes,
              _stream(stream, dev)))


# ----------------------------------------------------------------- activation

def _act(name: str) -> int:
    code = _ACT.get(name)
    if code is None:
        raise ValueError(f"act: {name!r}, expected {' or '.join(map(repr, _ACT))}")
    return code


def zero_activation_fp8(u: torch.Tensor, v: Optional[torch.Tensor], act: str, a: Optional[torch.Tensor] = None,
                        a8: Optional[Pair] = None, u8: Optional[Pair] = None, v8: Optional[Pair] = None,
                        stream=None) -> None:
    """a = act(u) * v (act(u) with v None; act "silu" or "gelu", its tanh form) in u's type
    and, in 8 bits, into a8; checkpoints of u and v into u8 and v8."""
    if u.dim() != 2:
        raise ValueError("u: matrix expected")
    (rows, cols), dev = u.shape, _current()
    if v is None and v8 is not None:
        raise ValueError("v8: there is no v")
    pu, ldu = _matrix(u, rows, cols, "u", _HALF, dev)
    dt = (u.dtype,)
    check("zero_activation_fp8",
          lib().zero_activation_fp8(
              pu, ldu, *_some(v, rows, cols, "v", dt, dev), _act(act), _TYPE[u.dtype], rows, cols,
              *_some(a, rows, cols, "a", dt, dev), _one_type(a8), _form(a8, rows, cols, "a8", _F8, dev),
              _form(u8, rows, cols, "u8", _E4M3, dev), _form(v8, rows, cols, "v8", _E4M3, dev), _stream(stream, dev)))


def zero_activation_backward_fp8(da: torch.Tensor, u: torch.Tensor, v: Optional[torch.Tensor], act: str,
                                 su: Optional[torch.Tensor] = None, sv: Optional[torch.Tensor] = None,
                                 du: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                                 du8: Optional[Pair] = None, dv8: Optional[Pair] = None,
                                 du8t: Optional[Pair] = None, dv8t: Optional[Pair] = None,
                                 a8t: Optional[Pair] = None, stream=None) -> None:
    """The gradients of zero_activation_fp8 from da: du and dv as halves, in 8 bits
    (du8, dv8) and, transposed, with blocks along the rows (du8t, dv8t); the
    activation again, transposed (a8t, E4M3).  u, v: what was kept, halves, or E4M3 with
    the scales su and sv."""
    if da.dim() != 2:
        raise ValueError("da: matrix expected")
    (rows, cols), dev = da.shape, _current()
    if v is None and any(t is not None for t in (sv, dv, dv8, dv8t)):
        raise ValueError("there is no v")
    if v is not None and (su is None) != (sv is None):
        raise ValueError("su and sv: both or neither expected")
    dt = da.dtype
    pda, ldda = _matrix(da, rows, cols, "da", _HALF, dev)
    check("zero_activation_backward_fp8",
          lib().zero_activation_backward_fp8(
              pda, ldda, *_kept(u, su, rows, cols, "u", dt, dev),
              *(_kept(v, sv, rows, cols, "v", dt, dev) if v is not None else (None, 0, None, 0)), _act(act),
              _TYPE[dt], rows, cols, *_some(du, rows, cols, "du", (dt,), dev),
              *_some(dv, rows, cols, "dv", (dt,), dev), _one_type(du8, dv8, du8t, dv8t),
              _form(du8, rows, cols, "du8", _F8, dev), _form(dv8, rows, cols, "dv8", _F8, dev),
              _form(du8t, cols, rows, "du8t", _F8, dev), _form(dv8t, cols, rows, "dv8t", _F8, dev),
              _form(a8t, cols, rows, "a8t", _E4M3, dev), _stream(stream, dev)))


# ----------------------------------------------------------------- reading back

def zero_fp8_restore(q: torch.Tensor, s: torch.Tensor, row: Optional[torch.Tensor] = None,
                     col: Optional[torch.Tensor] = None, x: Optional[torch.Tensor] = None,
                     t8: Optional[Pair] = None, stream=None) -> None:
    """q * s * row * col (a factor for each row, fp32, and each column) into x and,
    transposed, in 8 bits of q's type with blocks along q's rows, into t8."""
    if q.dim() != 2:
        raise ValueError("q: matrix expected")
    (rows, cols), dev = q.shape, _current()
    pq, ldq = _matrix(q, rows, cols, "q", _F8, dev)
    ps, lds = _matrix(s, _blocks(cols), rows, "s", _F32, dev)
    px, ldx = _some(x, rows, cols, "x", _FLOAT, dev)
    check("zero_fp8_restore",
          lib().zero_fp8_restore(
              pq, _TYPE[q.dtype], ldq, ps, lds, _vector(row, rows, "row", dev, torch.float32),
              _vector(col, cols, "col", dev), T_F32 if col is None else _type(col), rows, cols,
              px, T_F32 if x is None else _TYPE[x.dtype], ldx, _form(t8, cols, rows, "t8", (q.dtype,), dev),
              _stream(stream, dev)))
