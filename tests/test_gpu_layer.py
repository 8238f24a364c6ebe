"""What lies between a layer's products against plain 64-bit forms on the GPU.  The
bounds on errors are layer_reference's, derived beside each formula."""
import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from layer_reference import activation, check_form, check_half, form64, norms, norms_backward, value
from ops_reference import U, half_ulp

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
EPS = 1e-5


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, shape, dtype=F32, sigma=1.0, mean=0.0):
    return (torch.randn(shape, device="cuda", generator=gen(seed)) * sigma + mean).to(dtype)


def strided(x, pad, fill):
    """x as a view whose rows are `pad` elements further apart, the gaps filled."""
    if pad == 0:
        return x
    big = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=F32, device="cuda").to(x.dtype)
    big[:, :x.shape[1]] = x
    return big[:, :x.shape[1]]


def gaps_are(value_, *views):
    for v in views:
        assert (v._base[:, v.shape[1]:].float() == value_).all()


def gate_of(kind, rows, cols, dtype=F32, seed=77):
    shape = {"none": None, "one": (1,), "cols": (cols,), "rows": (rows, 1)}[kind]
    return None if shape is None else torch.sigmoid(normal(seed, shape)).to(dtype)


def pair(rows, cols, dtype=E4M3, pad=0):
    q, s = zs.fp8_empty(rows, cols, dtype)
    if pad:
        q = strided(torch.zeros(rows, cols, device="cuda").to(dtype), pad, 5.0)
        s = strided(torch.zeros(s.shape, device="cuda"), pad, 5.0)
    return q, s


def same(a, b):
    return torch.equal(a.float(), b.float()) if a.dtype in (E4M3, E5M2) else torch.equal(a, b)


# ----------------------------------------------------------------- norms, forward

WIDTHS = [1, 7, 16, 120, 128, 129, 200, 256, 257, 768, 1001, 2048, 2056, 4096, 4100, 5120, 8192, 8200, 16384, 16391, 20000]
KINDS = ["none", "one", "cols", "rows"]


def run_norms(o, x, w_pre, w_post, gate, scale, f8=E4M3, pad=0):
    rows, cols = o.shape
    out = dict(h=strided(torch.zeros_like(o), pad, 5.0), y=strided(torch.zeros_like(o), pad, 5.0),
               y8=pair(rows, cols, f8, pad), o8=pair(rows, cols, E4M3, pad), h8=pair(rows, cols, E4M3, pad),
               rstd_post=torch.full((rows,), 7.0, device="cuda"), rstd_pre=torch.full((rows,), 7.0, device="cuda"))
    zs.zero_gated_norms_fp8(o, x, w_pre, EPS, out["h"], w_post=w_post, gate=gate, scale=scale,
                            **{k: v for k, v in out.items() if k != "h"})
    return out


def check_norms(out, o, x, w_pre, w_post, gate, scale):
    want = norms(o, x, w_post, w_pre, gate, scale, EPS)
    check_half(out["h"], want["h"], want["eh"])
    check_half(out["y"], want["y"], want["ey"])
    check_form(*out["y8"], want["y"], want["ey"])
    check_form(*out["h8"], want["h"], want["eh"])
    assert ((out["rstd_pre"].double() - want["rh"]).abs() <= want["rh"] * (want["er"] + 4 * U)).all()
    if w_post is not None:
        assert ((out["rstd_post"].double() - want["ro"]).abs() <= want["ro"] * want["r"]).all()
    else:
        assert (out["rstd_post"] == 7.0).all()
    q, s = pair(*o.shape)
    zs.zero_fp8_quantize(o, q, s)
    assert same(q, out["o8"][0]) and torch.equal(s, out["o8"][1])  # the framework's own 8-bit form of o


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind", KINDS)
def test_norms(cols, kind):
    i = WIDTHS.index(cols) + KINDS.index(kind)
    rows = [3, 37, 1, 18][i % 4]
    dt, wt = [(BF16, F32), (F16, F16), (BF16, BF16), (F16, F32)][(i // 2) % 4]
    o, x = normal(cols, (rows, cols), dt, 3.0), normal(cols + 1, (rows, cols), dt)
    w_pre = normal(2, (cols,), wt, 0.2, 1.0)
    w_post = normal(3, (cols,), wt, 0.2, 1.0) if i % 3 else None
    gate, scale = gate_of(kind, rows, cols, wt), [1.0, 0.75, -2.0][i % 3]
    out = run_norms(o, x, w_pre, w_post, gate, scale, [E4M3, E5M2][i % 2])
    check_norms(out, o, x, w_pre, w_post, gate, scale)


@pytest.mark.parametrize("pad", [1, 8, 16])
@pytest.mark.parametrize("cols", [100, 264, 1000, 4096, 16400])
def test_norms_strides_leave_the_gaps(cols, pad):
    o = strided(normal(1, (5, cols), BF16), pad, float("nan"))
    x = strided(normal(2, (5, cols), BF16), pad, float("nan"))
    w = normal(3, (cols,), F32, 0.1, 1.0)
    out = run_norms(o, x, w, w, None, 1.0, E4M3, pad)
    check_norms(out, o, x, w, w, None, 1.0)
    gaps_are(5.0, out["h"], out["y"], *out["y8"], *out["o8"], *out["h8"])


@pytest.mark.parametrize("cols", [96, 1000, 4096, 16400])
@pytest.mark.parametrize("over", ["x", "o"])
def test_norms_in_place(cols, over):
    o, x = normal(1, (9, cols), F16), normal(2, (9, cols), F16)
    w = normal(3, (cols,), F16, 0.1, 1.0)
    want = run_norms(o, x, w, w, None, 0.5)
    y8 = pair(9, cols)
    h = {"x": x, "o": o}[over]
    zs.zero_gated_norms_fp8(o, x, w, EPS, h, w_post=w, scale=0.5, y8=y8)
    assert torch.equal(h, want["h"]) and same(y8[0], want["y8"][0]) and torch.equal(y8[1], want["y8"][1])


def test_norms_each_output_alone():
    rows, cols = 33, 1000
    o, x, w = normal(1, (rows, cols), BF16), normal(2, (rows, cols), BF16), normal(3, (cols,), BF16, 0.1, 1.0)
    want = run_norms(o, x, w, w, None, 1.0)
    for name in ("y", "y8", "o8", "h8", "rstd_post", "rstd_pre"):
        out = tuple(torch.empty_like(t) for t in want[name]) if name.endswith("8") else torch.empty_like(want[name])
        h = torch.empty_like(o)
        zs.zero_gated_norms_fp8(o, x, w, EPS, h, w_post=w, **{name: out})
        assert torch.equal(h, want["h"])
        for a, b in zip(out, want[name]) if isinstance(out, tuple) else [(out, want[name])]:
            assert same(a, b)


@pytest.mark.parametrize("cols", [100, 200, 1000, 16400])
def test_norms_rows_of_zeros_and_of_what_is_not_finite(cols):
    o, x = normal(1, (20, cols), BF16), normal(2, (20, cols), BF16)
    w = torch.ones(cols, device="cuda")
    o[3], x[3] = 0, 0
    o[5, 1], x[7, cols - 1], o[19, 0] = float("nan"), float("inf"), float("-inf")
    o[11], x[11] = 3e38, 0  # squares beyond fp32: the norm is 0
    out = run_norms(o, x, w, w, None, 1.0)
    assert (out["h"][3] == 0).all() and (out["y8"][0][3].float() == 0).all()
    bad = [5, 7, 19]
    good = [r for r in range(20) if r not in bad]
    v = out["y8"][0].float() * out["y8"][1].t().repeat_interleave(128, 1)[:, :cols]
    assert not v[[5, 19]].isfinite().any()  # a NaN, or an infinity that the norm behind the block makes one
    # an infinity in the stream: its norm is 1 / sqrt(inf) = 0, so its block is 0 * inf and the others are 0
    b = (cols - 1) // 128 * 128
    assert v[7, b:].isnan().all() and (v[7, :b] == 0).all()
    assert out["y"][good].float().isfinite().all() and v[good].isfinite().all()
    assert float(out["rstd_post"][11]) == 0.0 and (out["h"][11] == 0).all()


# ----------------------------------------------------------------- norms, backward

def run_backward(dy, dh, o, h, ro, rh, w_post, w_pre, gate, scale, so=None, sh=None, dwt=F32, ws=None, pad=0, add=None):
    rows, cols = dy.shape
    out = dict(d_o=strided(torch.zeros_like(dy), pad, 5.0), dx=strided(torch.zeros_like(dy), pad, 5.0))
    start = 0.0 if add is None else add
    out["dw_pre"] = torch.full((cols,), start, device="cuda", dtype=dwt)
    out["dw_post"] = torch.full((cols,), start, device="cuda", dtype=dwt) if w_post is not None else None
    out["dgate"] = torch.full(gate.shape, start, device="cuda", dtype=dwt) if gate is not None else None
    if ws is None:
        ws = torch.full((zs.zero_gated_norms_workspace_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    zs.zero_gated_norms_backward(dy, o, h, w_pre, rh, out["d_o"], out["dx"], ws, so=so, sh=sh, dh=dh, w_post=w_post,
                                 rstd_post=ro if w_post is not None else None, gate=gate, scale=scale,
                                 dw_pre=out["dw_pre"], dw_post=out["dw_post"], dgate=out["dgate"], add=add is not None)
    return out


def check_backward(out, dy, dh, o, h, ro, rh, w_post, w_pre, gate, scale, so=None, sh=None, start=0.0):
    want = norms_backward(dy, dh, value(o, so), value(h, sh), ro, rh, w_post, w_pre, gate, scale)
    check_half(out["dx"], want["dx"], want["dx_err"])
    check_half(out["d_o"], want["d_o"], want["d_o_err"])
    for name in ("dw_pre", "dw_post", "dgate"):
        got = out[name]
        if got is not None:
            kept = start if name != "dgate" or gate.shape != (dy.shape[0], 1) else 0.0
            w = want[name].reshape(got.shape) + kept
            err = want[name + "_err"].reshape(got.shape) + w.abs() * U
            assert ((got.double() - w).abs() <= err + half_ulp(w.abs() + err, got.dtype) * (1 + 1e-6)).all(), name


def backward_inputs(rows, cols, dt, wt, kind, post, s8, seed=0):
    o, h = normal(seed + 1, (rows, cols), dt, 2.0), normal(seed + 2, (rows, cols), dt)
    ro = torch.rsqrt(o.float().square().mean(1) + EPS)
    rh = torch.rsqrt(h.float().square().mean(1) + EPS)
    so = sh = None
    if s8:
        (o, so), (h, sh) = ((strided(q, 16 - q.shape[1] % 16, 5.0), s) for q, s in (form64(o.double(), E4M3), form64(h.double(), E4M3)))
    w_pre = normal(seed + 3, (cols,), wt, 0.2, 1.0)
    w_post = normal(seed + 4, (cols,), wt, 0.2, 1.0) if post else None
    dy, dh = normal(seed + 5, (rows, cols), dt), normal(seed + 6, (rows, cols), dt)
    return dict(dy=dy, dh=dh, o=o, h=h, ro=ro, rh=rh, w_post=w_post, w_pre=w_pre, gate=gate_of(kind, rows, cols, wt),
                so=so, sh=sh)


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind", KINDS)
def test_norms_backward(cols, kind, s8):
    i = WIDTHS.index(cols) + KINDS.index(kind)
    rows = [3, 700, 1, 45][i % 4]
    dt, wt = [(BF16, F32), (F16, F16), (BF16, BF16), (F16, F32)][(i // 2) % 4]
    a = backward_inputs(rows, cols, dt, wt, kind, i % 3 > 0, s8)
    if i % 5 == 0:
        a["dh"] = None
    scale = [1.0, 0.75, -2.0][i % 3]
    out = run_backward(scale=scale, dwt=[F32, BF16, F16][i % 3], **a)
    check_backward(out, scale=scale, **a)


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("rows,cols,kind", [(9000, 120, "one"), (5001, 256, "cols"), (4099, 768, "rows"), (2500, 4096, "cols"),
                                            (1300, 8192, "one"), (400, 8200, "cols")])
def test_norms_backward_many_rows(rows, cols, kind, s8):
    a = backward_inputs(rows, cols, BF16, F32, kind, True, s8)
    out = run_backward(scale=1.0, **a)
    check_backward(out, scale=1.0, **a)
    again = run_backward(scale=1.0, **a)
    for k in out:
        assert out[k] is None or torch.equal(out[k], again[k])  # the same bits again


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("pad", [1, 8, 16])
@pytest.mark.parametrize("cols", [72, 200, 1000, 4096, 8200])
def test_norms_backward_strides(cols, pad, s8):
    a = backward_inputs(21, cols, F16, F32, "cols", True, s8)
    for k in ("dy", "dh") + (() if s8 else ("o", "h")):
        a[k] = strided(a[k], pad, float("nan"))
    if s8:  # rows that no wide access takes
        a["o"], a["h"] = (strided(a[k].clone(), pad, 3.0) for k in ("o", "h"))
    out = run_backward(scale=1.0, pad=pad, **a)
    check_backward(out, scale=1.0, **a)
    gaps_are(5.0, out["d_o"], out["dx"])


@pytest.mark.parametrize("cols", [96, 1000, 4096, 8200])
@pytest.mark.parametrize("crossed", [False, True])
def test_norms_backward_in_place(cols, crossed):
    a = backward_inputs(50, cols, BF16, F32, "one", True, True)
    want = run_backward(scale=1.0, **a)
    d_o, dx = (a["dh"], a["dy"]) if crossed else (a["dy"], a["dh"])
    zs.zero_gated_norms_backward(a["dy"], a["o"], a["h"], a["w_pre"], a["rh"], d_o, dx, None, so=a["so"], sh=a["sh"],
                                 dh=a["dh"], w_post=a["w_post"], rstd_post=a["ro"], gate=a["gate"])
    assert torch.equal(d_o, want["d_o"]) and torch.equal(dx, want["dx"])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [0, 5])
def test_norms_backward_adds(kind, rows):
    a = backward_inputs(rows, 200, BF16, F32, kind, True, False)
    out = run_backward(scale=1.0, add=3.0, **a)
    check_backward(out, scale=1.0, start=3.0, **a)
    if rows == 0:
        out = run_backward(scale=1.0, **a)
        for k in ("dw_pre", "dw_post", "dgate"):
            assert out[k] is None or (out[k] == 0).all()


def test_norms_backward_of_a_gate_of_zero():
    """A gate that starts at 0 lets nothing through to the block and still learns."""
    a = backward_inputs(40, 300, BF16, F32, "cols", True, True)
    a["gate"].zero_()
    out = run_backward(scale=1.0, **a)
    check_backward(out, scale=1.0, **a)
    assert (out["d_o"] == 0).all() and (out["dw_post"] == 0).all() and (out["dgate"] != 0).all()


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_norms_gradients_against_differences(kind, post):
    """The loss sum(dy y) + sum(dh h) in 64 bits along a direction: (L(+t) - L(-t)) / 2t is off by t^2 times a third
    derivative (t = 1e-5: far below the rest).  What was kept is h in fp16, off by 2^-11 of itself, and so xh; a
    gradient's terms carry xh at most three times."""
    rows, cols, scale = 12, 96, 0.75
    a = backward_inputs(rows, cols, F16, F32, kind, post, False)
    o, x = a["o"], normal(9, (rows, cols), F16)
    w_pre, w_post, gate = a["w_pre"].double(), a["w_post"], a["gate"]
    got0 = norms(o, x, w_post, w_pre, gate, scale, EPS)
    ro, rh, h = got0["ro"].float(), got0["rh"].float(), got0["h"].to(F16)
    args = dict(a, o=o, h=h, ro=ro, rh=rh)
    out = run_backward(scale=scale, **args)
    size = norms_backward(a["dy"], a["dh"], o.double(), h.double(), ro, rh, w_post, a["w_pre"], gate, scale)

    def loss(o_, x_, wp, wo, g):
        n = norms(o_, x_, wo, wp, g, scale, EPS)
        return (a["dy"].double() * n["y"]).sum() + (a["dh"].double() * n["h"]).sum()

    base = [o.double(), x.double(), w_pre, None if w_post is None else w_post.double(), None if gate is None else gate.double()]
    for i, name in enumerate(("d_o", "dx", "dw_pre", "dw_post", "dgate")):
        if base[i] is None:
            continue
        d = normal(20 + i, tuple(base[i].shape)).double()
        t = 1e-5
        up, dn = (loss(*[b + sgn * t * d if k == i else b for k, b in enumerate(base)]) for sgn in (1, -1))
        diff = float((up - dn) / (2 * t))
        mine = float((out[name].double() * d).sum())
        r = 40 * U  # the errors' bounds are sizes times at least this
        err = size[name + "_err"].reshape(d.shape)
        tol = float(((err / r * 3 * 2 ** -11 + err + half_ulp(out[name].double(), out[name].dtype)) * d.abs()).sum())
        assert abs(diff - mine) <= tol + 1e-6 * abs(diff)


# ----------------------------------------------------------------- activation

ACT_SHAPES = [(1, 1), (1, 128), (3, 7), (127, 129), (128, 128), (130, 255), (33, 1000), (300, 264), (5, 4104)]


@pytest.mark.parametrize("rows,cols", ACT_SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
def test_activation(rows, cols, act, gated):
    i = ACT_SHAPES.index((rows, cols)) + (act == "gelu") + gated
    dt, f8 = [(BF16, E4M3), (F16, E5M2), (BF16, E5M2), (F16, E4M3)][i % 4]
    u, v = normal(1, (rows, cols), dt, 4.0), normal(2, (rows, cols), dt) if gated else None
    u[0, 0], u[-1, -1] = -100.0, 60.0
    a, a8, u8 = torch.empty_like(u), pair(rows, cols, f8), pair(rows, cols)
    v8 = pair(rows, cols) if gated else None
    zs.zero_activation_fp8(u, v, act, a=a, a8=a8, u8=u8, v8=v8)
    want = activation(u.double(), v.double() if gated else None, act)
    check_half(a, want["a"], want["ae"])
    check_form(*a8, want["a"], want["ae"])
    for x, got in ((u, u8), (v, v8)):
        if x is not None:
            q, s = pair(rows, cols)
            zs.zero_fp8_quantize(x, q, s)
            assert same(q, got[0]) and torch.equal(s, got[1])
    alone = torch.empty_like(u)
    zs.zero_activation_fp8(u, v, act, a=alone)
    assert torch.equal(alone, a)
    over = u.clone()
    zs.zero_activation_fp8(over, v, act, a=over)
    assert torch.equal(over, a)


@pytest.mark.parametrize("pad", [1, 8])
def test_activation_strides_leave_the_gaps(pad):
    u, v = (strided(normal(i, (70, 200), BF16), pad, float("nan")) for i in (1, 2))
    a, a8, u8, v8 = strided(torch.zeros(70, 200, device="cuda", dtype=BF16), pad, 5.0), pair(70, 200, E4M3, pad), \
        pair(70, 200, E4M3, pad), pair(70, 200, E4M3, pad)
    zs.zero_activation_fp8(u, v, "silu", a=a, a8=a8, u8=u8, v8=v8)
    want = activation(u.double(), v.double(), "silu")
    check_half(a, want["a"], want["ae"])
    check_form(*a8, want["a"], want["ae"])
    check_form(*v8, v.double(), torch.zeros(70, 200, device="cuda", dtype=torch.float64))
    gaps_are(5.0, a, *a8, *u8, *v8)


def test_activation_of_extreme_values():
    u = torch.tensor([[0.0, -0.0, 1e-38, -1e-38, 88.0, -88.0, 104.0, -104.0, 3e38, -3e38, 1e-3, -1e30]], device="cuda").to(BF16)
    for act in ("silu", "gelu"):
        a, du, da = torch.empty_like(u), torch.empty_like(u), torch.ones_like(u)
        zs.zero_activation_fp8(u, None, act, a=a)
        want = activation(u.double(), None, act)
        check_half(a, want["a"], want["ae"])
        zs.zero_activation_backward_fp8(da, u, None, act, du=du)
        slope = torch.where(u.double().abs() > 200, (u > 0).double(), want["slope"])  # 0 times a large number
        err = torch.where(u.double().abs() > 200, 4 * U + 0 * slope, want["se"])
        check_half(du, slope, err)
    u[0, 3] = float("nan")
    zs.zero_activation_fp8(u, None, "gelu", a=a)
    assert a[0, 3].isnan() and a[0, :3].isfinite().all()


def run_act_backward(da, u, v, act, su, sv, f8, pad=0, half=True):
    rows, cols = da.shape
    o = dict(du=strided(torch.zeros_like(da), pad, 5.0) if half else None, du8=pair(rows, cols, f8, pad),
             du8t=pair(cols, rows, f8, pad), a8t=pair(cols, rows, E4M3, pad))
    if v is not None:
        o.update(dv=strided(torch.zeros_like(da), pad, 5.0) if half else None, dv8=pair(rows, cols, f8, pad),
                 dv8t=pair(cols, rows, f8, pad))
    zs.zero_activation_backward_fp8(da, u, v, act, su=su, sv=sv, **o)
    return o


def check_act_backward(o, da, u, v, act, su, sv):
    da, u64 = da.double(), value(u, su)
    v64 = value(v, sv) if v is not None else None
    want = activation(u64, v64, act)
    vv = torch.ones_like(u64) if v is None else v64
    grads = [("du", da * vv * want["slope"], (da * vv).abs() * (want["se"] + want["slope"].abs() * 6 * U))]
    if v is not None:
        grads.append(("dv", da * want["f"], da.abs() * (want["fe"] + want["f"].abs() * 6 * U)))
    for name, x, err in grads + [("a", want["a"], want["ae"] + want["a"].abs() * 4 * U)]:
        if o.get(name) is not None:
            check_half(o[name], x, err)
        if name + "8" in o:
            check_form(*o[name + "8"], x, err)
        # through bf16: half a step, relative 2^-8, and half of its smallest number
        check_form(*o[name + "8t"], x.t(), err.t(), err.t() + (x.t().abs() + err.t()) * 2 ** -8 + 2.0 ** -134)


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("rows,cols", ACT_SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
def test_activation_backward(rows, cols, act, gated, s8):
    i = ACT_SHAPES.index((rows, cols)) + (act == "gelu") + gated
    dt, f8 = [(BF16, E4M3), (F16, E5M2), (BF16, E5M2), (F16, E4M3)][i % 4]
    u, v = normal(1, (rows, cols), dt, 4.0), normal(2, (rows, cols), dt)
    da, su, sv = normal(3, (rows, cols), dt), None, None
    if s8:
        (u, su), (v, sv) = ((strided(q, 16 - q.shape[1] % 16, 5.0), s) for q, s in (form64(u.double(), E4M3), form64(v.double(), E4M3)))
    if not gated:
        v = sv = None
    o = run_act_backward(da, u, v, act, su, sv, f8)
    check_act_backward(o, da, u, v, act, su, sv)
    for name in list(o):  # each output alone gives the same bits
        one = tuple(torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda") for t in o[name]) \
            if isinstance(o[name], tuple) else torch.empty_like(o[name])
        zs.zero_activation_backward_fp8(da, u, v, act, su=su, sv=sv, **{name: one})
        for a, b in zip(one, o[name]) if isinstance(one, tuple) else [(one, o[name])]:
            assert same(a, b), name


@pytest.mark.parametrize("pad", [1, 8])
def test_activation_backward_strides_and_in_place(pad):
    da, u, v = (strided(normal(i, (150, 200), F16), pad, float("nan")) for i in (1, 2, 3))
    o = run_act_backward(da, u, v, "silu", None, None, E5M2, pad)
    check_act_backward(o, da, u, v, "silu", None, None)
    for t in o.values():
        gaps_are(5.0, *(t if isinstance(t, tuple) else (t,)))
    over = da.clone()
    dv = torch.empty_like(over)
    zs.zero_activation_backward_fp8(over, u, v, "silu", du=over, dv=dv)
    assert torch.equal(over, o["du"]) and torch.equal(dv, o["dv"])


def test_activation_backward_passes_on_what_is_not_finite():
    da, u = normal(1, (140, 300), BF16), normal(2, (140, 300), BF16)
    da[5, 130] = float("inf")
    o = run_act_backward(da, u, None, "silu", None, None, E5M2)
    v = o["du8"][0].float() * o["du8"][1].t().repeat_interleave(128, 1)[:, :300]
    vt = (o["du8t"][0].float() * o["du8t"][1].t().repeat_interleave(128, 1)[:, :140]).t()
    for got, rows, cols in ((v, slice(5, 6), slice(128, 256)), (vt, slice(0, 128), slice(130, 131))):
        hit = torch.zeros(140, 300, dtype=torch.bool, device="cuda")
        hit[rows, cols] = True
        assert not got[hit].isfinite().any() and got[~hit].isfinite().all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_gradients_against_differences(act):
    """(f(+t) - f(-t)) / 2t in 64 bits, off by t^2 times a third derivative below 1."""
    u, v, da = normal(1, (40, 100), F16, 3.0), normal(2, (40, 100), F16), normal(3, (40, 100), F16)
    o = run_act_backward(da, u, v, act, None, None, E4M3)
    t = 1e-4
    up, dn = (activation(u.double() + s * t, v.double(), act)["a"] for s in (1, -1))
    du = da.double() * (up - dn) / (2 * t)
    want = activation(u.double(), v.double(), act)
    check_half(o["du"], du, (da.double() * v.double()).abs() * (want["se"] + 1e-6) + du.abs() * 8 * U)
    up, dn = (activation(u.double(), v.double() + s * t, act)["a"] for s in (1, -1))
    dv = da.double() * (up - dn) / (2 * t)
    check_half(o["dv"], dv, da.double().abs() * (want["fe"] + 1e-9) + dv.abs() * 8 * U)


# ----------------------------------------------------------------- reading back

@pytest.mark.parametrize("f8", [E4M3, E5M2])
@pytest.mark.parametrize("rows,cols", ACT_SHAPES + [(256, 384), (1000, 16)])
def test_restore(rows, cols, f8):
    i = rows + cols
    q, s = form64(normal(1, (rows, cols)).double() * torch.exp(normal(2, (rows, 1))).double(), f8)
    q = strided(q, 16 - cols % 16, 5.0) if i % 3 else q.contiguous()
    row = torch.exp(normal(3, (rows,))) if i % 2 else None
    col = normal(4, (cols,), [F32, BF16, F16][i % 3], 0.3, 1.0) if i % 5 else None
    want = value(q, s)
    if row is not None:
        want = want * row.double()[:, None]
    if col is not None:
        want = want * col.double()
    err = want.abs() * 3 * U
    for xt in (F16, BF16, F32):
        x, t8 = torch.empty(rows, cols, dtype=xt, device="cuda"), pair(cols, rows, f8)
        zs.zero_fp8_restore(q, s, row=row, col=col, x=x, t8=t8)
        check_half(x, want, err)
        check_form(*t8, want.t(), err.t())
    alone, x1 = pair(cols, rows, f8), torch.empty_like(x)
    zs.zero_fp8_restore(q, s, row=row, col=col, t8=alone)
    zs.zero_fp8_restore(q, s, row=row, col=col, x=x1)
    assert same(alone[0], t8[0]) and torch.equal(alone[1], t8[1]) and torch.equal(x, x1)


def test_restore_strides_and_what_is_not_finite():
    q, s = form64(normal(1, (130, 200)).double(), E4M3)
    s[1, 3] = float("inf")
    q[3, 128:] = float("nan")
    x, t8 = strided(torch.zeros(130, 200, device="cuda", dtype=BF16), 3, 5.0), pair(200, 130, E4M3, 3)
    zs.zero_fp8_restore(strided(q, 3, 5.0), s, x=x, t8=t8)
    gaps_are(5.0, x, *t8)
    assert x[3, 128:].isnan().all() and x[3, :128].isfinite().all() and x[4:].isfinite().all()
    v = t8[0].float() * t8[1].t().repeat_interleave(128, 1)[:, :130]
    assert not v[128:, :128].isfinite().any() and v[:128].isfinite().all() and v[128:, 128:].isfinite().all()
    clean = value(q, s)[:, :128]
    check_form(t8[0][:128], t8[1][:, :128], clean.t(), clean.t().abs() * 3 * U)


# ----------------------------------------------------------------- streams and graphs

def test_other_streams_and_graphs():
    """On a stream of its own, and captured: two graphs that share a workspace, replayed
    one after the other on new inputs."""
    rows, cols = 200, 1000
    a = backward_inputs(rows, cols, BF16, F32, "cols", True, True)
    b = backward_inputs(rows, cols, BF16, F32, "cols", True, True, seed=50)
    want_a, want_b = run_backward(scale=1.0, **a), run_backward(scale=1.0, **b)
    ws = torch.empty(zs.zero_gated_norms_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_backward(scale=1.0, ws=ws, **a)
    torch.cuda.current_stream().wait_stream(side)
    assert all(got[k] is None or torch.equal(got[k], want_a[k]) for k in got)
    static = {k: v.clone() if v is not None else None for k, v in a.items()}
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_backward(scale=1.0, ws=ws, **static))
        graphs.append(g)
    for src, want in ((a, want_a), (b, want_b)):
        for k, v in static.items():
            if v is not None:
                v.copy_(src[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got in outs:
            assert all(got[k] is None or torch.equal(got[k], want[k]) for k in got)


def test_empty():
    z = torch.empty(0, 64, device="cuda", dtype=BF16)
    w = torch.ones(64, device="cuda")
    zs.zero_gated_norms_fp8(z, z, w, EPS, z.clone(), w_post=w, y8=pair(0, 64))
    zs.zero_activation_fp8(z, z, "silu", a8=pair(0, 64))
    zs.zero_activation_backward_fp8(z, z, z, "silu", du8t=pair(64, 0))
    zs.zero_fp8_restore(*pair(0, 64), t8=pair(64, 0))
    torch.cuda.synchronize()
