"""Cases of the operators behind and ahead of a layer's products in 8 bits (norms with gate and
residual scale, activations, 8-bit checkpoints) for timing and comparison.

``own`` false: the operators in plain torch operations, in 32 bits.  ``own``
true: the calls a user makes of zero_partitioned_mixed_step_gb300.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
TINY = 2.0 ** -126  # the smallest scale of a block
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
K = math.sqrt(2.0 / math.pi)  # of gelu's tanh form


def listed():
    return [
        # Between two blocks of a decoder of width 4096, 8192 tokens: the norm behind the block, a
        # gate for each channel, the stream, the norm ahead of the next block's products in 8 bits,
        # and what the backward pass needs, in 8 bits.
        dict(name="norms 8192x4096 gate cols", op="norms", rows=8192, cols=4096, dtype="bf16", wt="fp32", gate="cols",
             post=True, scale=1.0, fp8="e4m3", y=False, saved="e4m3"),
        # Width 768 (12 layers), 16384 tokens, one learned number as the gate, fp16.
        dict(name="norms 16384x768 gate one", op="norms", rows=16384, cols=768, dtype="fp16", wt="fp16", gate="one",
             post=True, scale=0.8, fp8="e4m3", y=True, saved="e4m3"),
        # Seven tokens of an odd width, a gate for each token, nothing saved: latency.
        dict(name="norms 7x1001 gate rows", op="norms", rows=7, cols=1001, dtype="bf16", wt="bf16", gate="rows",
             post=True, scale=1.0, fp8="e4m3", y=True, saved="half"),
        # The gradients of the first, from the 8-bit checkpoints.
        dict(name="norms backward 8192x4096 gate cols", op="norms_backward", rows=8192, cols=4096, dtype="bf16",
             wt="fp32", gate="cols", post=True, scale=1.0, dh=True, saved="e4m3"),
        # A width between the powers of two, halves saved, no norm behind the block, a gate for each token.
        dict(name="norms backward 4099x2304 gate rows", op="norms_backward", rows=4099, cols=2304, dtype="fp16",
             wt="fp16", gate="rows", post=False, scale=0.8, dh=True, saved="half"),
        # The feed-forward's gated activation, 8192 tokens: its 8-bit output and both inputs saved in 8 bits.
        dict(name="activation 8192x14336 gated silu", op="act", rows=8192, cols=14336, dtype="bf16", act="silu",
             gated=True, fp8="e4m3", a=False, saved=True),
        # Sixteen tokens, nothing saved: latency.
        dict(name="activation 16x14336 gated silu", op="act", rows=16, cols=14336, dtype="bf16", act="silu",
             gated=True, fp8="e4m3", a=False, saved=False),
        # Its gradients from the checkpoints, in the forms that the products of the inputs' and the
        # weights' gradients take, and the transposed activation for the last weight's.
        dict(name="activation backward 8192x14336 gated silu", op="act_backward", rows=8192, cols=14336, dtype="bf16",
             act="silu", gated=True, fp8="e5m2", saved=True, half=False),
        # An odd number of tokens, no gate, gelu, the gradient as halves too.
        dict(name="activation backward 1021x2056 gelu", op="act_backward", rows=1021, cols=2056, dtype="fp16",
             act="gelu", gated=False, fp8="e4m3", saved=True, half=True),
        # The transposed operand of a weight's gradient from the stream's checkpoint: the norm's row and
        # column factors applied on the way.
        dict(name="restore 8192x4096 transposed", op="restore", rows=8192, cols=4096, fp8="e4m3", row=True, col=True,
             out="none", trans=True),
        # A whole feed-forward activation read back as halves, one factor for each row.
        dict(name="restore 8192x14336 bf16", op="restore", rows=8192, cols=14336, fp8="e4m3", row=True, col=False,
             out="bf16", trans=False),
        # Both, of an odd size.
        dict(name="restore 301x769 both", op="restore", rows=301, cols=769, fp8="e5m2", row=False, col=True,
             out="fp16", trans=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norms", "norms", "norms_backward", "norms_backward", "act", "act_backward", "act_backward", "restore"])
    half = rng.choice(["bf16", "fp16"])
    fp8 = rng.choice(["e4m3", "e4m3", "e5m2"])
    if op in ("norms", "norms_backward"):
        cols = _log(rng, 16, 16384)
        c = dict(op=op, rows=_log(rng, 1, min(65536, 8192 * 4096 // cols)), cols=cols, dtype=half,
                 wt=rng.choice([half, "fp32"]), gate=rng.choice(["none", "one", "cols", "rows"]),
                 post=rng.random() < 0.7, scale=rng.choice([1.0, 0.8]), saved=rng.choice(["e4m3", "e4m3", "half"]))
        return dict(c, fp8=fp8, y=rng.random() < 0.4) if op == "norms" else dict(c, dh=rng.random() < 0.8)
    cols = _log(rng, 1, 16384)
    rows = _log(rng, 1, min(65536, 8192 * 14336 // cols))
    if op == "restore":
        trans = rng.random() < 0.6
        return dict(op=op, rows=rows, cols=cols, fp8=fp8, row=rng.random() < 0.5, col=rng.random() < 0.5,
                    out=rng.choice(["none", "bf16", "fp16", "fp32"] if trans else ["bf16", "fp16", "fp32"]), trans=trans)
    c = dict(op=op, rows=rows, cols=cols, dtype=half, act=rng.choice(["silu", "gelu"]), gated=rng.random() < 0.7,
             fp8=fp8)
    if op == "act":
        return dict(c, a=rng.random() < 0.3, saved=rng.random() < 0.7)
    return dict(c, saved=rng.random() < 0.7, half=rng.random() < 0.3)


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFF)


def _normal(g, shape, sigma=1.0, mean=0.0):
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(mean, sigma, generator=g)


def _up(n, m):
    return (n + m - 1) // m * m


def _padded(rows, cols, dtype):
    """Rows of `cols` elements whose stride is a multiple of 16 bytes."""
    step = 16 // torch.empty(0, dtype=dtype).element_size()
    return torch.zeros(rows, _up(cols, step), device="cuda", dtype=dtype)[:, :cols]


def _pair(rows, cols, fp8):
    """An 8-bit matrix and its scales, one for each 1x128 block."""
    return _padded(rows, cols, F8[fp8]), torch.zeros(_up(cols, BLOCK) // BLOCK, rows, device="cuda")


def _in(x, dtype):
    out = _padded(*x.shape, dtype)
    out.copy_(x)
    return out


def _tokens(g, rows, cols):
    """Activations: normal, each row with its own size, a few channels much larger."""
    row = torch.exp(_normal(g, (rows, 1), 0.5))
    col = torch.exp(_normal(g, (1, cols), 0.7))
    return _normal(g, (rows, cols)).mul_(row).mul_(col)


def _checkpoint(x):
    """x in E4M3 with a scale for each 1x128 block."""
    q, s = _quantize(x.float(), "e4m3")
    return _in(q.float(), F8["e4m3"]), s


def prepare(case, seed):
    g, op, r, k = _gen(seed), case["op"], case["rows"], case["cols"]
    if op in ("norms", "norms_backward"):
        dt, wt = DT[case["dtype"]], DT[case["wt"]]
        st = dict(case, o=_in(_tokens(g, r, k), dt), x=_in(_tokens(g, r, k), dt),
                  w_pre=_normal(g, (k,), 0.1, 1.0).to(wt),
                  w_post=_normal(g, (k,), 0.1, 1.0).to(wt) if case["post"] else None, gate_=None)
        shape = {"none": None, "one": (1,), "cols": (k,), "rows": (r, 1)}[case["gate"]]
        if shape is not None:
            st["gate_"] = torch.sigmoid(_normal(g, shape)).to(wt)
        if op == "norms":
            e4 = case["saved"] == "e4m3"
            st.update(h=_padded(r, k, dt), yo=_padded(r, k, dt) if case["y"] else None, y8=_pair(r, k, case["fp8"]),
                      o8=_pair(r, k, "e4m3") if e4 else None, h8=_pair(r, k, "e4m3") if e4 else None,
                      rstd_post=torch.zeros(r, device="cuda") if case["post"] else None,
                      rstd_pre=torch.zeros(r, device="cuda"))
            return st
        st["rstd_post"] = torch.rsqrt(st["o"].float().square().mean(1) + EPS) if case["post"] else None
        st["rstd_pre"] = torch.rsqrt(st["x"].float().square().mean(1) + EPS)
        st["o"], st["so"] = _checkpoint(st["o"]) if case["saved"] == "e4m3" else (st["o"], None)
        st["h"], st["sh"] = _checkpoint(st["x"]) if case["saved"] == "e4m3" else (st["x"], None)
        del st["x"]
        st.update(dy=_in(_normal(g, (r, k), 1e-2), dt), dh_=_in(_normal(g, (r, k), 1e-2), dt) if case["dh"] else None,
                  d_o=_padded(r, k, dt), dx=_padded(r, k, dt), dw_pre=torch.zeros(k, device="cuda"),
                  dw_post=torch.zeros(k, device="cuda") if case["post"] else None,
                  dgate=torch.zeros(shape, device="cuda") if shape is not None else None)
        return st
    if op in ("act", "act_backward"):
        dt = DT[case["dtype"]]
        st = dict(case, u=_in(_tokens(g, r, k), dt), v=_in(_tokens(g, r, k), dt) if case["gated"] else None)
        if op == "act":
            st.update(a_=_padded(r, k, dt) if case["a"] else None, a8=_pair(r, k, case["fp8"]),
                      u8=_pair(r, k, "e4m3") if case["saved"] else None,
                      v8=_pair(r, k, "e4m3") if case["saved"] and case["gated"] else None)
            return st
        st["su"] = st["sv"] = None
        if case["saved"]:
            st["u"], st["su"] = _checkpoint(st["u"])
            if case["gated"]:
                st["v"], st["sv"] = _checkpoint(st["v"])
        st["da"] = _in(_normal(g, (r, k), 1e-2), dt)
        for n in ("u", "v")[:2 if case["gated"] else 1]:
            st["d" + n] = _padded(r, k, dt) if case["half"] else None
            st["d" + n + "8"], st["d" + n + "8t"] = _pair(r, k, case["fp8"]), _pair(k, r, case["fp8"])
        st["a8t"] = _pair(k, r, "e4m3")
        return st
    q, s = _pair(r, k, case["fp8"])
    q.copy_(_normal(g, (r, k), QMAX[case["fp8"]] / 4.0).clamp_(-QMAX[case["fp8"]], QMAX[case["fp8"]]).to(q.dtype))
    s.copy_(torch.exp(_normal(g, tuple(s.shape), 0.7)) * (2.0 / QMAX[case["fp8"]]))
    return dict(case, q=q, s=s, r_=torch.exp(_normal(g, (r,), 0.3)) if case["row"] else None,
                c_=_normal(g, (k,), 0.1, 1.0) if case["col"] else None,
                x=_padded(r, k, DT[case["out"]]) if case["out"] != "none" else None,
                t8=_pair(k, r, case["fp8"]) if case["trans"] else None)


# ----------------------------------------------------------------- plain forms

def _block_amax(x):
    """[rows, cols] -> largest magnitude of each 1x128 block, [cols/128, rows]."""
    r, k = x.shape
    return torch.nn.functional.pad(x.abs(), (0, -k % BLOCK)).view(r, -1, BLOCK).amax(2).t()


def _spread(s, cols):
    """Scales [cols/128, rows] at each element of [rows, cols]."""
    return s.t().repeat_interleave(BLOCK, 1)[:, :cols]


def _quantize(x, fp8):
    s = (_block_amax(x) / QMAX[fp8]).clamp_min(TINY)
    return (x / _spread(s, x.shape[1])).to(F8[fp8]), s.contiguous()


def _both(name, x, fp8):
    """A matrix's 8-bit form as two outputs."""
    q, s = _quantize(x, fp8)
    return {name: q, name + " scales": s}


def _value(q, s):
    return q.float() if s is None else q.float() * _spread(s, q.shape[1])


def _factor(t):
    return 1.0 if t is None else t.float()


def _sigmoid_of(u, act):
    """(sigmoid, the derivative of its argument) of u * sigmoid(z(u))."""
    if act == "silu":
        return torch.sigmoid(u), 1.0
    return torch.sigmoid(2.0 * K * (u + 0.044715 * u * u * u)), 2.0 * K * (1.0 + 3.0 * 0.044715 * u * u)


def _plain(s):
    op = s["op"]
    if op == "norms":
        o, x, out = s["o"].float(), s["x"].float(), {}
        n = o
        if s["post"]:
            out["rstd_post"] = torch.rsqrt(o.square().mean(1) + EPS)
            n = o * out["rstd_post"][:, None] * s["w_post"].float()
        h = s["scale"] * x + _factor(s["gate_"]) * n
        out["rstd_pre"] = torch.rsqrt(h.square().mean(1) + EPS)
        y = h * out["rstd_pre"][:, None] * s["w_pre"].float()
        out["h"] = h.to(s["x"].dtype)
        out.update(_both("y8", y, s["fp8"]))
        if s["y"]:
            out["y"] = y.to(s["x"].dtype)
        if s["saved"] == "e4m3":
            out.update(_both("o8", o, "e4m3"))
            out.update(_both("h8", h, "e4m3"))
        return out
    if op == "norms_backward":
        dy, gate, a = s["dy"].float(), _factor(s["gate_"]), _factor(s["w_post"])
        xh = _value(s["h"], s["sh"]) * s["rstd_pre"][:, None]
        xo = _value(s["o"], s["so"])
        if s["post"]:
            xo = xo * s["rstd_post"][:, None]
        g = dy * s["w_pre"].float()
        dh = s["rstd_pre"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["dh"]:
            dh = dh + s["dh_"].float()
        d_o = dh * gate * a
        if s["post"]:
            d_o = s["rstd_post"][:, None] * (d_o - xo * (d_o * xo).mean(1, keepdim=True))
        out = {"d_o": d_o.to(s["dy"].dtype), "dx": (s["scale"] * dh).to(s["dy"].dtype), "dw_pre": (dy * xh).sum(0)}
        if s["post"]:
            out["dw_post"] = (gate * dh * xo).sum(0)
        if s["gate"] != "none":
            dg = dh * xo * a
            out["dgate"] = dg.sum(0) if s["gate"] == "cols" else dg.sum(1, keepdim=True) if s["gate"] == "rows" \
                else dg.sum(1).sum().reshape(1)
        return out
    if op == "act":
        u = s["u"].float()
        a = u * _sigmoid_of(u, s["act"])[0] * _factor(s["v"])
        out = _both("a8", a, s["fp8"])
        if s["a"]:
            out["a"] = a.to(s["u"].dtype)
        if s["saved"]:
            out.update(_both("u8", u, "e4m3"))
            if s["gated"]:
                out.update(_both("v8", s["v"].float(), "e4m3"))
        return out
    if op == "act_backward":
        u, da = _value(s["u"], s["su"]), s["da"].float()
        v = _value(s["v"], s["sv"]) if s["gated"] else 1.0
        sig, dz = _sigmoid_of(u, s["act"])
        act = u * sig
        du = da * v * (sig + act * (1.0 - sig) * dz)
        out = _both("du8", du, s["fp8"])
        out.update(_both("du8t", du.t(), s["fp8"]))
        out.update(_both("a8t", (act * v).t(), "e4m3"))
        if s["half"]:
            out["du"] = du.to(s["da"].dtype)
        if s["gated"]:
            dv = da * act
            out.update(_both("dv8", dv, s["fp8"]))
            out.update(_both("dv8t", dv.t(), s["fp8"]))
            if s["half"]:
                out["dv"] = dv.to(s["da"].dtype)
        return out
    x = _value(s["q"], s["s"])
    if s["row"]:
        x = x * s["r_"][:, None]
    if s["col"]:
        x = x * s["c_"]
    out = {"x": x.to(s["x"].dtype)} if s["out"] != "none" else {}
    if s["trans"]:
        out.update(_both("t8", x.t(), s["fp8"]))
    return out


# ----------------------------------------------------------------- the framework's calls

def _named(s, *names):
    """The outputs of these names that this case has, 8-bit matrices as two."""
    out = {}
    for n in names:
        t = s.get(n)
        if isinstance(t, tuple):
            out[n], out[n + " scales"] = t
        elif t is not None:
            out[{"yo": "y", "a_": "a"}.get(n, n)] = t
    return out


def _framework(s):
    import zero_partitioned_mixed_step_gb300 as zs
    op = s["op"]
    if op == "norms":
        zs.zero_gated_norms_fp8(s["o"], s["x"], s["w_pre"], EPS, s["h"], w_post=s["w_post"], gate=s["gate_"],
                                scale=s["scale"], y=s["yo"], y8=s["y8"], o8=s["o8"], h8=s["h8"],
                                rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
        return _named(s, "h", "yo", "y8", "o8", "h8", "rstd_post", "rstd_pre")
    if op == "norms_backward":
        if "ws" not in s:  # a user's program makes it once
            s["ws"] = torch.empty(zs.zero_gated_norms_workspace_bytes(s["rows"], s["cols"]), device="cuda",
                                  dtype=torch.uint8)
        zs.zero_gated_norms_backward(s["dy"], s["o"], s["h"], s["w_pre"], s["rstd_pre"], s["d_o"], s["dx"], s["ws"],
                                     so=s["so"], sh=s["sh"], dh=s["dh_"], w_post=s["w_post"],
                                     rstd_post=s["rstd_post"], gate=s["gate_"], scale=s["scale"], dw_pre=s["dw_pre"],
                                     dw_post=s["dw_post"], dgate=s["dgate"])
        return _named(s, "d_o", "dx", "dw_pre", "dw_post", "dgate")
    if op == "act":
        zs.zero_activation_fp8(s["u"], s["v"], s["act"], a=s["a_"], a8=s["a8"], u8=s["u8"], v8=s["v8"])
        return _named(s, "a_", "a8", "u8", "v8")
    if op == "act_backward":
        zs.zero_activation_backward_fp8(s["da"], s["u"], s["v"], s["act"], su=s["su"], sv=s["sv"], du=s["du"],
                                        dv=s.get("dv"), du8=s["du8"], dv8=s.get("dv8"), du8t=s["du8t"],
                                        dv8t=s.get("dv8t"), a8t=s["a8t"])
        return _named(s, "du", "dv", "du8", "dv8", "du8t", "dv8t", "a8t")
    zs.zero_fp8_restore(s["q"], s["s"], row=s["r_"], col=s["c_"], x=s["x"], t8=s["t8"])
    return _named(s, "x", "t8")


def run(state):
    return _framework(state) if own else _plain(state)


# ----------------------------------------------------------------- bytes and operations

def work(case):
    op, r, k = case["op"], case["rows"], case["cols"]
    kb, rb = _up(k, BLOCK) // BLOCK, _up(r, BLOCK) // BLOCK
    form, formt = r * k + 4 * kb * r, r * k + 4 * rb * k  # an 8-bit form and its scales, the transposed one
    if op in ("norms", "norms_backward"):
        e, post = SIZE[case["dtype"]], case["post"]
        gate = {"none": 0, "one": 1, "cols": k, "rows": r}[case["gate"]]
        vec = SIZE[case["wt"]] * (k * (2 if post else 1) + gate)
        if op == "norms":
            return {"bytes": r * k * e * (4 if case["y"] else 3) + form * (3 if case["saved"] == "e4m3" else 1) + vec
                    + 4 * r * (2 if post else 1), "flops": 16 * r * k}
        saved = form if case["saved"] == "e4m3" else r * k * e
        return {"bytes": r * k * e * (4 if case["dh"] else 3) + 2 * saved + vec + 4 * r * (2 if post else 1)
                + 4 * (k * (2 if post else 1) + gate), "flops": 24 * r * k}
    if op == "restore":
        return {"bytes": form + (r * k * SIZE[case["out"]] if case["out"] != "none" else 0)
                + (formt if case["trans"] else 0) + 4 * (r if case["row"] else 0) + 4 * (k if case["col"] else 0),
                "flops": 4 * r * k}
    e, n = SIZE[case["dtype"]], 2 if case["gated"] else 1
    if op == "act":
        return {"bytes": r * k * e * (n + (1 if case["a"] else 0)) + form * (1 + (n if case["saved"] else 0)),
                "flops": 10 * r * k}
    return {"bytes": r * k * e * (1 + (n if case["half"] else 0)) + n * (form if case["saved"] else r * k * e)
            + n * (form + formt) + formt, "flops": 24 * r * k}


# ----------------------------------------------------------------- the definitions in 64 bits

def _blocks64(name, x, fp8, qmax=QMAX):
    """x / s before its rounding to 8 bits, and s, one block of columns after the other."""
    q, s = torch.empty_like(x), []
    for part, to in zip(x.split(BLOCK, 1), q.split(BLOCK, 1)):
        s.append(torch.clamp(part.abs().max(1).values / qmax[fp8], min=TINY))
        torch.div(part, s[-1][:, None], out=to)
    return {name: q, name + " scales": torch.stack(s)}


def _value64(q, s):
    x = q.double()
    if s is not None:
        for part, f in zip(x.split(BLOCK, 1), s.double()):
            part.mul_(f[:, None])
    return x


def _root64(x):
    return (torch.einsum("rk,rk->r", x, x) / x.shape[1] + EPS) ** -0.5


def _act64(u, act):
    if act == "silu":
        return u * torch.sigmoid(u)
    return 0.5 * u * (1.0 + torch.tanh(K * (u + 0.044715 * u ** 3)))


def exact(case, seed):
    s, op, k = prepare(case, seed), case["op"], case["cols"]
    ones = torch.ones(k, device="cuda", dtype=torch.float64)
    if op in ("norms", "norms_backward"):
        w, wp = s["w_pre"].double(), s["w_post"].double() if case["post"] else ones
        gate = torch.ones(1, device="cuda", dtype=torch.float64) if s["gate_"] is None else s["gate_"].double()
    if op == "norms":
        o, out = s["o"].double(), {}
        h = case["scale"] * s["x"].double()
        if case["post"]:
            out["rstd_post"] = _root64(o)
            h += torch.einsum("rk,r,k->rk", o, out["rstd_post"], wp) * gate
        else:
            h += o * gate
        out["rstd_pre"] = _root64(h)
        out["h"], y = h, torch.einsum("rk,r,k->rk", h, out["rstd_pre"], w)
        out.update(_blocks64("y8", y, case["fp8"]))
        if case["y"]:
            out["y"] = y
        if case["saved"] == "e4m3":
            out.update(_blocks64("o8", o, "e4m3"))
            out.update(_blocks64("h8", h, "e4m3"))
        return out
    if op == "norms_backward":
        dy, h, o = s["dy"].double(), _value64(s["h"], s["sh"]), _value64(s["o"], s["so"])
        rh = s["rstd_pre"].double()
        ro = s["rstd_post"].double() if case["post"] else torch.ones_like(rh)
        along = torch.einsum("rk,rk,k->r", dy, h, w) * rh ** 3 / k
        dh = torch.einsum("rk,k,r->rk", dy, w, rh) - h * along[:, None]
        if case["dh"]:
            dh += s["dh_"].double()
        d_o = dh * gate * wp * ro[:, None]
        if case["post"]:
            d_o -= o * (torch.einsum("rk,rk->r", d_o, o) * ro ** 2 / k)[:, None]
        out = {"dx": dh * case["scale"], "d_o": d_o, "dw_pre": torch.einsum("rk,rk,r->k", dy, h, rh)}
        dn = dh * o * ro[:, None]  # of gate * w_post
        if case["post"]:
            out["dw_post"] = (dn * gate).sum(0)
        if case["gate"] != "none":
            dg = dn @ wp if case["gate"] != "cols" else dn.sum(0) * wp
            out["dgate"] = dg if case["gate"] == "cols" else dg[:, None] if case["gate"] == "rows" else dg.sum().reshape(1)
        return out
    if op == "act":
        u = s["u"].double()
        a = _act64(u, case["act"])
        if case["gated"]:
            a = a * s["v"].double()
        out = _blocks64("a8", a, case["fp8"])
        if case["a"]:
            out["a"] = a
        if case["saved"]:
            out.update(_blocks64("u8", u, "e4m3"))
            if case["gated"]:
                out.update(_blocks64("v8", s["v"].double(), "e4m3"))
        return out
    if op == "act_backward":
        with torch.enable_grad():
            u = _value64(s["u"], s["su"]).requires_grad_()
            leaves = [u]
            a = _act64(u, case["act"])
            if case["gated"]:
                leaves.append(_value64(s["v"], s["sv"]).requires_grad_())
                a = a * leaves[1]
            grads = torch.autograd.grad(a, leaves, s["da"].double())
        out = _blocks64("a8t", a.detach().t().contiguous(), "e4m3")
        for n, d in zip(("du", "dv"), grads):
            out.update(_blocks64(n + "8", d, case["fp8"]))
            out.update(_blocks64(n + "8t", d.t().contiguous(), case["fp8"]))
            if case["half"]:
                out[n] = d
        return out
    x = _value64(s["q"], s["s"])
    if case["row"]:
        x = torch.einsum("rk,r->rk", x, s["r_"].double())
    if case["col"]:
        x = torch.einsum("rk,k->rk", x, s["c_"].double())
    out = {"x": x} if case["out"] != "none" else {}
    if case["trans"]:
        out.update(_blocks64("t8", x.t().contiguous(), case["fp8"]))
    return out
