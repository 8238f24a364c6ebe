"""What lies between a layer's products where it can go wrong: rows that start on wide boundaries
and end inside a unit, offsets beyond 32 bits, calls side by side, several turns of a CTA."""
import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from layer_reference import check_form, form64, value
from ops_reference import U
from test_gpu_layer import (BF16, E4M3, E5M2, EPS, F16, F32, backward_inputs, check_act_backward, check_backward,
                            check_norms, gate_of, normal, pair, run_act_backward, run_backward, run_norms, same)

pytestmark = pytest.mark.gpu


def aligned(x, fill=float("nan")):
    """x in rows that start on 32-byte boundaries, what lies between them filled."""
    step = 32 // x.element_size()
    rows, cols = x.shape
    big = torch.full((rows, (cols + step) // step * step), fill, dtype=F32, device="cuda").to(x.dtype)
    big[:, :cols] = x
    return big[:, :cols]


def gaps(*views):
    return torch.cat([v._base[:, v.shape[1]:].float().flatten() for v in views])


def wide_pair(rows, cols, dtype=E4M3):
    return aligned(torch.zeros(rows, cols, device="cuda").to(dtype), 5.0), zs.fp8_empty(rows, cols, dtype)[1]


# every remainder of 8, in each way that rows are shared out
RAGGED = [9, 42, 91, 131, 174, 255, 301, 612, 1021, 1998, 2055, 2308, 2555, 3334, 4093, 4097, 6002, 8191, 9003, 16379, 16390]


@pytest.mark.parametrize("cols", RAGGED)
def test_norms_rows_that_end_inside_a_unit(cols):
    rows, i = 29, RAGGED.index(cols)
    dt, kind = (BF16, F16)[i % 2], ("cols", "rows", "one", "none")[i % 4]
    o, x = aligned(normal(cols, (rows, cols), dt, 2.0)), aligned(normal(cols + 1, (rows, cols), dt))
    w_pre, w_post = normal(2, (cols,), F32, 0.2, 1.0), normal(3, (cols,), F32, 0.2, 1.0) if i % 3 else None
    gate = gate_of(kind, rows, cols)
    out = dict(h=aligned(torch.zeros_like(o), 5.0), y=aligned(torch.zeros_like(o), 5.0),
               y8=wide_pair(rows, cols, (E4M3, E5M2)[i % 2]), o8=wide_pair(rows, cols), h8=wide_pair(rows, cols),
               rstd_post=torch.full((rows,), 7.0, device="cuda"), rstd_pre=torch.empty(rows, device="cuda"))
    zs.zero_gated_norms_fp8(o, x, w_pre, EPS, out["h"], w_post=w_post, gate=gate, scale=0.75,
                            **{k: v for k, v in out.items() if k != "h"})
    check_norms(out, o, x, w_pre, w_post, gate, 0.75)
    assert (gaps(out["h"], out["y"], out["y8"][0], out["o8"][0], out["h8"][0]) == 5.0).all()
    packed = run_norms(o.contiguous(), x.contiguous(), w_pre, w_post, gate, 0.75, out["y8"][0].dtype)
    for k in out:  # how rows lie changes no bit
        for a, b in zip(out[k], packed[k]) if isinstance(out[k], tuple) else [(out[k], packed[k])]:
            assert same(a, b), k


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("cols", RAGGED)
def test_norms_backward_rows_that_end_inside_a_unit(cols, s8):
    i = RAGGED.index(cols)
    a = backward_inputs(31, cols, (BF16, F16)[i % 2], F32, ("cols", "rows", "one", "none")[i % 4], i % 3 > 0, s8)
    for k in ("dy", "dh", "o", "h"):
        a[k] = aligned(a[k], 3.0 if a[k].dtype == E4M3 else float("nan"))
    d_o, dx = aligned(torch.zeros_like(a["dy"]), 5.0), aligned(torch.zeros_like(a["dy"]), 5.0)
    out = run_backward(scale=0.75, **a)
    check_backward(out, scale=0.75, **a)
    zs.zero_gated_norms_backward(a["dy"], a["o"], a["h"], a["w_pre"], a["rh"], d_o, dx, None, so=a["so"], sh=a["sh"],
                                 dh=a["dh"], w_post=a["w_post"], rstd_post=a["ro"], gate=a["gate"], scale=0.75)
    # the sums over a row are the same ones, so the gradients are
    assert torch.equal(d_o, out["d_o"]) and torch.equal(dx, out["dx"]) and (gaps(d_o, dx) == 5.0).all()


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 9), (7, 131), (135, 42), (257, 255), (130, 1021), (300, 2052)])
def test_activation_rows_that_end_inside_a_unit(rows, cols, gated, s8):
    u, v, da = (aligned(normal(i, (rows, cols), BF16, 2.0)) for i in (1, 2, 3))
    a, a8, u8, v8 = aligned(torch.zeros_like(u), 5.0), wide_pair(rows, cols, E5M2), wide_pair(rows, cols), wide_pair(rows, cols)
    if not gated:
        v = v8 = None
    zs.zero_activation_fp8(u, v, "gelu", a=a, a8=a8, u8=u8, v8=v8)
    b, b8, c8 = torch.empty_like(u.contiguous()), pair(rows, cols, E5M2), pair(rows, cols)
    zs.zero_activation_fp8(u.contiguous(), v.contiguous() if gated else None, "gelu", a=b, a8=b8, u8=c8)
    assert torch.equal(a, b) and same(a8[0], b8[0]) and torch.equal(a8[1], b8[1]) and same(u8[0], c8[0])
    assert (gaps(a, a8[0], u8[0], *([v8[0]] if gated else [])) == 5.0).all()
    su = sv = None
    if s8:
        (u, su), (v, sv) = u8, v8 if gated else (None, None)
    o = dict(du=aligned(torch.zeros_like(da), 5.0), du8=wide_pair(rows, cols, E5M2), du8t=wide_pair(cols, rows, E5M2),
             a8t=wide_pair(cols, rows))
    if gated:
        o.update(dv=aligned(torch.zeros_like(da), 5.0), dv8=wide_pair(rows, cols, E5M2), dv8t=wide_pair(cols, rows, E5M2))
    zs.zero_activation_backward_fp8(da, u, v, "gelu", su=su, sv=sv, **o)
    check_act_backward(o, da, u, v, "gelu", su, sv)
    assert (gaps(*(t[0] if isinstance(t, tuple) else t for t in o.values())) == 5.0).all()


@pytest.mark.parametrize("f8", [E4M3, E5M2])
@pytest.mark.parametrize("rows,cols", [(1, 9), (7, 131), (135, 42), (257, 255), (130, 1021)])
def test_restore_rows_that_end_inside_a_unit(rows, cols, f8):
    q, s = form64(normal(1, (rows, cols)).double(), f8)
    q = aligned(q, 3.0)
    row, col = torch.exp(normal(3, (rows,))), normal(4, (cols,), BF16, 0.3, 1.0)
    x, t8 = aligned(torch.zeros(rows, cols, device="cuda", dtype=F16), 5.0), wide_pair(cols, rows, f8)
    zs.zero_fp8_restore(q, s, row=row, col=col, x=x, t8=t8)
    want = value(q, s) * row.double()[:, None] * col.double()
    check_form(*t8, want.t(), want.t().abs() * 3 * U)
    assert (gaps(x, t8[0]) == 5.0).all()
    y = torch.empty(rows, cols, device="cuda", dtype=F16)
    zs.zero_fp8_restore(q.contiguous(), s, row=row, col=col, x=y)
    assert torch.equal(x, y)


# ----------------------------------------------------------------- offsets beyond 32 bits

def test_norms_beyond_32_bits():
    """2.4e9 elements: the last rows are those of a call on them alone."""
    rows, cols, m = 590_000, 4096, 64
    o, x, dy = (torch.zeros(rows, cols, device="cuda", dtype=BF16) for _ in range(3))
    for i, t in enumerate((o, x, dy)):
        t[-m:] = normal(i, (m, cols), BF16)
    w = normal(5, (cols,), F32, 0.1, 1.0)
    h, y8, o8, h8 = torch.empty_like(o), pair(rows, cols), pair(rows, cols), pair(rows, cols)
    ro, rh = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zs.zero_gated_norms_fp8(o, x, w, EPS, h, w_post=w, y8=y8, o8=o8, h8=h8, rstd_post=ro, rstd_pre=rh)
    want = run_norms(o[-m:].clone(), x[-m:].clone(), w, w, None, 1.0)
    assert torch.equal(h[-m:], want["h"]) and torch.equal(rh[-m:], want["rstd_pre"])
    for a, b in ((y8, want["y8"]), (o8, want["o8"]), (h8, want["h8"])):
        assert same(a[0][-m:], b[0]) and torch.equal(a[1][:, -m:], b[1])
    d_o, dx = x, h  # places that are no longer needed
    zs.zero_gated_norms_backward(dy, o8[0], h8[0], w, rh, d_o, dx, None, so=o8[1], sh=h8[1], w_post=w, rstd_post=ro)
    few, fx = torch.empty(m, cols, device="cuda", dtype=BF16), torch.empty(m, cols, device="cuda", dtype=BF16)
    zs.zero_gated_norms_backward(dy[-m:], want["o8"][0], want["h8"][0], w, rh[-m:], few, fx, None, so=want["o8"][1],
                                 sh=want["h8"][1], w_post=w, rstd_post=ro[-m:])
    assert torch.equal(d_o[-m:], few) and torch.equal(dx[-m:], fx)


def test_activation_and_restore_beyond_32_bits():
    rows, cols, m = 300_032, 8192, 128
    u, da = (torch.zeros(rows, cols, device="cuda", dtype=BF16) for _ in range(2))
    for i, t in enumerate((u, da)):
        t[-m:] = normal(i, (m, cols), BF16)
    a8, u8 = pair(rows, cols), pair(rows, cols)
    zs.zero_activation_fp8(u, None, "silu", a8=a8, u8=u8)
    fa, fu = pair(m, cols), pair(m, cols)
    zs.zero_activation_fp8(u[-m:], None, "silu", a8=fa, u8=fu)
    for a, b in ((a8, fa), (u8, fu)):
        assert same(a[0][-m:], b[0]) and torch.equal(a[1][:, -m:], b[1])
    du8, du8t, x8t = pair(rows, cols, E5M2), pair(cols, rows, E5M2), pair(cols, rows)
    zs.zero_activation_backward_fp8(da, u8[0], None, "silu", su=u8[1], du8=du8, du8t=du8t)
    few, fewt = pair(m, cols, E5M2), pair(cols, m, E5M2)
    zs.zero_activation_backward_fp8(da[-m:], fu[0], None, "silu", su=fu[1], du8=few, du8t=fewt)
    assert same(du8[0][-m:], few[0]) and torch.equal(du8[1][:, -m:], few[1])
    assert same(du8t[0][:, -m:], fewt[0]) and torch.equal(du8t[1][-1:], fewt[1])
    zs.zero_fp8_restore(*u8, x=da, t8=x8t)
    fx, ft = torch.empty(m, cols, device="cuda", dtype=BF16), pair(cols, m)
    zs.zero_fp8_restore(*fu, x=fx, t8=ft)
    assert torch.equal(da[-m:], fx) and same(x8t[0][:, -m:], ft[0]) and torch.equal(x8t[1][-1:], ft[1])


# ----------------------------------------------------------------- several turns, calls side by side

@pytest.mark.parametrize("rows,cols", [(20_011, 100), (10_007, 200), (3_001, 500), (1_999, 2400), (701, 4096), (333, 8192)])
def test_norms_several_turns(rows, cols):
    o, x, w = normal(1, (rows, cols), BF16), normal(2, (rows, cols), BF16), normal(3, (cols,), F32, 0.1, 1.0)
    for w_post in (w, None):
        out = run_norms(o, x, w, w_post, None, 1.0)
        check_norms(out, o, x, w, w_post, None, 1.0)


@pytest.mark.parametrize("rows,cols", [(3000, 4000), (20_000, 130)])
def test_activation_several_turns(rows, cols):
    u, v, da = (normal(i, (rows, cols), F16) for i in (1, 2, 3))
    o = run_act_backward(da, u, v, "silu", None, None, E4M3)
    check_act_backward(o, da, u, v, "silu", None, None)
    a, a8 = torch.empty_like(u), pair(rows, cols)
    zs.zero_activation_fp8(u, v, "silu", a=a, a8=a8)
    q, s = pair(rows, cols)
    zs.zero_fp8_quantize(a, q, s)
    err = a.double().abs() * 2 ** -10  # a is a8's value rounded to fp16
    check_form(*a8, a.double(), err + 2.0 ** -24)


def test_calls_side_by_side():
    """Four streams at once, each with its own workspace."""
    rows, cols = 900, 2304
    args = [backward_inputs(rows, cols, BF16, F32, "cols", True, True, seed=10 * i) for i in range(4)]
    want = [run_backward(scale=1.0, **a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    got = [None] * 4
    for _ in range(5):
        for i, (st, a) in enumerate(zip(streams, args)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got[i] = run_backward(scale=1.0, **a)
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(g[k] is None or torch.equal(g[k], w[k]) for k in g)


# ----------------------------------------------------------------- checkpoints of every half

@pytest.mark.parametrize("dtype", [BF16, F16])
def test_checkpoints_of_every_largest_value(dtype):
    """Each finite value of the type as a block's largest, 127 smaller ones beside it: the scales are
    zero_fp8_quantize's bit for bit, and so are the values (of bf16 below 2^117, from where on
    either's quotients may be an fp32 unit off)."""
    big = torch.arange(0x7F80 if dtype == BF16 else 0x7C00, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    part = torch.rand(big.numel(), 128, device="cuda", generator=g, dtype=torch.float64) * 2 - 1
    u = (big.double()[:, None] * part).to(dtype)
    u[:, 5] = -big
    u8, want = pair(*u.shape), pair(*u.shape)
    zs.zero_activation_fp8(u, None, "silu", u8=u8)
    zs.zero_fp8_quantize(u, *want)
    assert torch.equal(u8[1], want[1])
    low = big.double() < 2.0 ** 117
    assert torch.equal(u8[0][low].float(), want[0][low].float())
    q, s = u8[0][~low].double(), u8[1][0][~low].double()[:, None]
    assert ((q - u[~low].double() / s).abs() <= (u[~low].double() / s).abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10 + 2.0 ** -20).all()


@pytest.mark.parametrize("cols", [4600, 9000])
@pytest.mark.parametrize("over", ["x", "o"])
def test_long_norms_in_place(cols, over):
    o, x = normal(1, (9, cols), BF16), normal(2, (9, cols), BF16)
    w = normal(3, (cols,), F32, 0.1, 1.0)
    want = run_norms(o, x, w, w, None, 0.5)
    y8, h = pair(9, cols), {"x": x, "o": o}[over]
    zs.zero_gated_norms_fp8(o, x, w, EPS, h, w_post=w, scale=0.5, y8=y8)
    assert torch.equal(h, want["h"]) and same(y8[0], want["y8"][0]) and torch.equal(y8[1], want["y8"][1])


def test_forward_and_backward_in_one_graph():
    """A block's end, forward and backward, and the activation's, captured once and replayed on new inputs."""
    rows, cols = 300, 1000
    w = normal(3, (cols,), F32, 0.1, 1.0)
    o, x, u, v, dy = (normal(i, (rows, cols), BF16) for i in range(5))
    ws = torch.empty(zs.zero_gated_norms_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    h, d_o, dx, du, dv = (torch.empty_like(o) for _ in range(5))
    o8, h8, y8, u8, v8, a8, t8 = (*(pair(rows, cols) for _ in range(6)), pair(cols, rows))
    ro, rh, dw = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")

    def chain():
        zs.zero_gated_norms_fp8(o, x, w, EPS, h, w_post=w, y8=y8, o8=o8, h8=h8, rstd_post=ro, rstd_pre=rh)
        zs.zero_activation_fp8(u, v, "silu", a8=a8, u8=u8, v8=v8)
        zs.zero_activation_backward_fp8(dy, u8[0], v8[0], "silu", su=u8[1], sv=v8[1], du=du, dv=dv)
        zs.zero_fp8_restore(*h8, row=rh, col=w, t8=t8)
        zs.zero_gated_norms_backward(dy, o8[0], h8[0], w, rh, d_o, dx, ws, so=o8[1], sh=h8[1], dh=du, w_post=w,
                                     rstd_post=ro, dw_pre=dw)

    def outputs():
        return [t.float().clone() for t in (h, d_o, dx, du, dv, dw, *y8, *a8, *t8)]

    chain()
    first = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for seed in (0, 40):
        for i, t in enumerate((o, x, u, v, dy)):
            t.copy_(normal(seed + i, (rows, cols), BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = outputs()
        chain()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outputs()))
        assert seed or all(torch.equal(a, b) for a, b in zip(got, first))
