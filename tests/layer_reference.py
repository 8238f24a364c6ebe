"""Plain 64-bit forms of what lies between a layer's products, with bounds on what
fp32 arithmetic may be off by, for the GPU tests.

u = 2^-24 is an fp32 operation's relative error; a sum of n terms in any order is off
by at most (n - 1) u times the sum of their magnitudes."""
import math

import torch

from ops_reference import QMAX, TINY, U, at_elements, block_amax, blocks, half_ulp

K = math.sqrt(2.0 / math.pi)


def row_terms(cols):
    """Additions on a term's way into a row's sum: a thread's own, the lanes', the warps'."""
    return 16 + cols // 1024 + 10


def check_form(q, s, x64, err, err_q=None):
    """(q, s) is the 8-bit form of x64, known to within err before the cast (err_q: for q alone)."""
    err_q = err if err_q is None else err_q
    want = torch.clamp(block_amax(x64, False) / QMAX[q.dtype], min=TINY)
    assert s.shape == want.shape
    assert ((s.double() - want).abs() <= want * 2 * U + block_amax(err, False) / QMAX[q.dtype]).all()
    spread = at_elements(s, *x64.shape, False)
    y, e = x64 / spread, err_q / spread
    off = (q.double() - y).abs()
    assert (off <= half_ulp(y.abs() + e, q.dtype) * (1 + 1e-6) + e + y.abs() * 3 * U).all()


def check_half(got, want, err):
    assert ((got.double() - want).abs() <= err + half_ulp(want.abs() + err, got.dtype) * (1 + 1e-6)).all()


def value(q, s):
    return q.double() if s is None else q.double() * at_elements(s, *q.shape, False)


def form64(x64, dtype):
    """x64's 8-bit form, scales rounded to fp32."""
    s = torch.clamp(block_amax(x64, False) / QMAX[dtype], min=TINY).float()
    return (x64 / at_elements(s, *x64.shape, False)).float().to(dtype), s


def norms(o, x, w_post, w_pre, gate, scale, eps):
    """h, y, ro, rh of the forward pass and bounds on each one's error."""
    o, x = o.double(), x.double()
    cols = o.shape[1]
    r = (row_terms(cols) + 8) * U
    g = 1.0 if gate is None else gate.double()
    ro = torch.ones(o.shape[0], dtype=torch.float64, device=o.device)
    n = o
    if w_post is not None:
        ro = 1.0 / torch.sqrt((o * o).mean(1) + eps)
        n = o * ro[:, None] * w_post.double()
    h = scale * x + g * n
    eh = ((scale * x).abs() + (g * n).abs()) * (r + 8 * U)
    rh = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    er = r + (h.abs() * eh).mean(1) * rh ** 2 + (eh * eh).mean(1) * rh ** 2
    y = h * rh[:, None] * w_pre.double()
    ey = y.abs() * (er[:, None] + 4 * U) + eh * (rh * (1 + er))[:, None] * w_pre.double().abs()
    return dict(h=h, eh=eh, ro=ro, rh=rh, er=er, r=r, y=y, ey=ey)


def norms_backward(dy, dh, o, h, ro, rh, w_post, w_pre, gate, scale):
    """Gradients from what was kept (64-bit values o and h, fp32 ro and rh) and bounds on their errors."""
    dy, cols, rows = dy.double(), dy.shape[1], dy.shape[0]
    r = (row_terms(cols) + 12) * U
    rh = rh.double()[:, None]
    xh = h * rh
    xo = o * ro.double()[:, None] if w_post is not None else o
    w, a = w_pre.double(), torch.ones(cols, dtype=torch.float64, device=dy.device) if w_post is None else w_post.double()
    gt = torch.ones(1, dtype=torch.float64, device=dy.device) if gate is None else gate.double()
    g = dy * w
    m = (g * xh).mean(1, keepdim=True)
    dH = rh * (g - xh * m)
    size = rh * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        dH, size = dH + dh.double(), size + dh.double().abs()
    out = dict(dx=scale * dH, dx_err=abs(scale) * size * r)
    G, Gs = gt * a * dH, (gt * a).abs() * size
    if w_post is not None:
        f = ro.double()[:, None]
        out["d_o"] = f * (G - xo * (G * xo).mean(1, keepdim=True))
        out["d_o_err"] = f * (Gs + xo.abs() * (Gs * xo.abs()).mean(1, keepdim=True)) * 3 * r
    else:
        out["d_o"], out["d_o_err"] = G, Gs * 2 * r
    rr = (rows + 20) * U  # any order of the rows
    out["dw_pre"], out["dw_pre_err"] = (dy * xh).sum(0), (dy * xh).abs().sum(0) * rr
    dn, dns = dH * xo, size * xo.abs()
    out["dw_post"], out["dw_post_err"] = (gt * dn).sum(0), (gt.abs() * dns).sum(0) * (rr + 2 * r)
    if gate is not None:
        dg, dgs = dn * a, dns * a.abs()
        if gate.shape == (rows, 1):
            out["dgate"], out["dgate_err"] = dg.sum(1, keepdim=True), dgs.sum(1, keepdim=True) * 3 * r
        elif gate.numel() == 1:
            out["dgate"], out["dgate_err"] = dg.sum().reshape(1), dgs.sum().reshape(1) * (rr + 3 * r)
        else:
            out["dgate"], out["dgate_err"] = dg.sum(0), dgs.sum(0) * (rr + 2 * r)
    return out


def activation(u, v, act):
    """a = act(u) v, act(u), its slope, and bounds.  CUDA's fast exponential is off by 2 + 1.16 |z|
    units, the fast quotient by 2, z by 4 roundings; the sigmoid is 0 below 2^-126."""
    if act == "silu":
        z, dz = u, torch.ones_like(u)
    else:
        z, dz = 2 * K * (u + 0.044715 * u ** 3), 2 * K * (1 + 3 * 0.044715 * u ** 2)
    sig = torch.sigmoid(z)
    rel = (16 + 8 * z.abs().clamp_max(400.0)) * U
    tiny = 2.0 ** -125
    f = u * sig
    slope = sig + f * torch.sigmoid(-z) * dz
    fe = f.abs() * rel + u.abs() * tiny
    # 1 - sig is off by sig's error; beyond |z| = 88 the sigmoid is 0 or 1
    se = (sig + (f * dz).abs()) * (rel + 8 * U) + (1 + (u * dz).abs()) * tiny + (f * dz).abs() * sig * rel
    vv = torch.ones_like(u) if v is None else v
    return dict(f=f, fe=fe, slope=slope, se=se, a=f * vv, ae=fe * vv.abs() + (f * vv).abs() * 2 * U)
