"""The 8-bit forms of what lies between a layer's products where their values are known exactly, and what
is not finite in them."""
import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from layer_reference import check_form, value
from test_gpu_layer import BF16, E4M3, E5M2, F16, F32, backward_inputs, gen, pair, run_backward, strided

pytestmark = pytest.mark.gpu


def as_bytes(q):
    return q.contiguous().view(torch.uint8)


def same_form(a, b):
    """The same bytes and scales, those of NaN too."""
    return torch.equal(as_bytes(a[0]), as_bytes(b[0])) and torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


def whole(seed, shape, low, high):
    return torch.randint(low, high + 1, shape, device="cuda", generator=gen(seed)).double()


def exact_act(rows, cols, dtype, s8, gated, seed=0):
    """(da, u, v, su, sv) and the 64-bit (du, dv, a).  u >= 32, where exp(-u) < 2^-25: in fp32 the sigmoid
    is 1, silu's and gelu's slopes are 1, and du = da v, dv = da u, a = u v are products of numbers of
    at most 6 bits, which fp32 holds and 8 bits of fraction do not."""
    da = (whole(seed + 1, (rows, cols), -63, 63) / 64).to(dtype)
    if s8:  # 4 bits each, and a power of two for each block
        u, v = (whole(seed + 2, (rows, cols), 8, 15) * 4).to(E4M3), whole(seed + 3, (rows, cols), -15, 15).to(E4M3)
        u, v = (strided(q, 16 - cols % 16, 5.0) for q in (u, v))
        su, sv = (2.0 ** whole(seed + i, ((cols + 127) // 128, rows), 0, 2).float() for i in (4, 5))
    else:
        u, v = whole(seed + 2, (rows, cols), 32, 63).to(dtype), (whole(seed + 3, (rows, cols), -63, 63) / 8).to(dtype)
        su = sv = None
    if not gated:
        v = sv = None
    u64, v64 = value(u, su), torch.ones_like(da, dtype=torch.float64) if v is None else value(v, sv)
    return (da, u, v, su, sv), (da.double() * v64, da.double() * u64, u64 * v64)


SHAPES = [(1, 1), (7, 131), (128, 128), (130, 255), (300, 264), (260, 1000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_transposed_gradients_are_rounded_once(rows, cols, s8, gated):
    """Off by half a step of the 8 bits and the quotient's units, and by nothing else."""
    i = SHAPES.index((rows, cols))
    dtype, f8, act = (BF16, F16)[i % 2], (E4M3, E5M2)[(i + s8) % 2], ("silu", "gelu")[(i + gated) % 2]
    (da, u, v, su, sv), (du, dv, a) = exact_act(rows, cols, dtype, s8, gated)
    out = dict(du8t=pair(cols, rows, f8), a8t=pair(cols, rows))
    if gated:
        out["dv8t"] = pair(cols, rows, f8)
    zs.zero_activation_backward_fp8(da, u, v, act, su=su, sv=sv, **out)
    for name, x in (("du8t", du), ("dv8t", dv), ("a8t", a)):
        if name in out:
            check_form(*out[name], x.t(), torch.zeros_like(x).t())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cols", [100, 128, 300, 1000, 5000, 16400])
def test_checkpoints_of_what_is_not_finite(cols, dtype):
    """o8, u8 and v8 are zero_fp8_quantize's form, byte for byte, in blocks that hold an infinity or a NaN."""
    rows = 9
    x = (torch.randn(rows, cols, device="cuda", generator=gen(1)) * 3).to(dtype)
    x[1, 3], x[2, cols - 1], x[3, cols // 2] = float("inf"), float("-inf"), float("nan")
    x[4, 0], x[4, cols - 1], x[5] = float("inf"), float("nan"), float("inf")
    x[6, ::2], x[6, 1::2] = -0.0, float("inf")
    want, o8, u8, v8 = (pair(rows, cols) for _ in range(4))
    zs.zero_fp8_quantize(x, *want)
    w = torch.ones(cols, device="cuda")
    zs.zero_gated_norms_fp8(x, torch.zeros_like(x), w, 1e-5, torch.empty_like(x), o8=o8)
    zs.zero_activation_fp8(x, x, "silu", u8=u8, v8=v8)
    alone = pair(rows, cols)
    zs.zero_activation_fp8(x, None, "gelu", u8=alone)
    assert all(same_form(got, want) for got in (o8, u8, v8, alone))


def quantized(x64, dtype):
    """zero_fp8_quantize's form of values that fp32 holds, and its transpose's."""
    (rows, cols), x = x64.shape, x64.float().contiguous()
    assert (x.double() == x64).all()
    q, t = pair(rows, cols, dtype), pair(cols, rows, dtype)
    zs.zero_fp8_quantize(x, *q, *t)
    return q, t


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_forms_of_computed_values_are_the_quotients(rows, cols, s8, gated):
    """What is computed in fp32 is divided as zero_fp8_quantize divides it: the same bytes, also where a quotient is
    the middle of two 8-bit values, which numbers of few bits often have."""
    i = SHAPES.index((rows, cols))
    dtype, f8, act = (F16, BF16)[i % 2], (E5M2, E4M3)[(i + s8) % 2], ("gelu", "silu")[(i + gated) % 2]
    args, values = exact_act(rows, cols, dtype, s8, gated, 10)
    da, u, v, su, sv = args
    out = dict(du8=pair(rows, cols, f8), du8t=pair(cols, rows, f8), a8t=pair(cols, rows))
    if gated:
        out.update(dv8=pair(rows, cols, f8), dv8t=pair(cols, rows, f8))
    zs.zero_activation_backward_fp8(da, u, v, act, su=su, sv=sv, **out)
    for name, x in zip(("du", "dv", "a"), values):
        along, across = quantized(x, E4M3 if name == "a" else f8)
        for got, want in ((name + "8", along), (name + "8t", across)):
            assert got not in out or same_form(out[got], want), got
    if not s8:
        a8 = pair(rows, cols, f8)
        zs.zero_activation_fp8(u, v, act, a8=a8)
        assert same_form(a8, quantized(values[2], f8)[0])


@pytest.mark.parametrize("f8", [E4M3, E5M2])
@pytest.mark.parametrize("cols", [64, 256, 1024, 2048, 4096, 8192, 16384, 32768])
def test_norms_forms_of_computed_values_are_the_quotients(cols, f8):
    """Whole numbers make h exact.  A row whose elements are all +-2^k has a mean square of 4^k, exact as cols is a
    power of two, and so with eps = 0 y = +-w."""
    rows = 24
    o, x = whole(1, (rows, cols), -31, 31).to(BF16), whole(2, (rows, cols), -31, 31).to(BF16)
    w = (whole(3, (cols,), 1, 63) * whole(4, (cols,), 1, 63)).float()
    h8, y8, h = pair(rows, cols), pair(rows, cols, f8), torch.empty_like(o)
    gate = 2.0 ** whole(5, (rows, 1), -2, 2).float()
    zs.zero_gated_norms_fp8(o, x, w, 0.0, h, gate=gate, scale=0.5, h8=h8)
    assert same_form(h8, quantized(0.5 * x.double() + gate.double() * o.double(), E4M3)[0])
    sign = whole(6, (rows, cols), 0, 1) * 2 - 1
    x = (sign * 2.0 ** whole(7, (rows, 1), -3, 3)).to(BF16)
    zs.zero_gated_norms_fp8(torch.zeros_like(x), x, w, 0.0, h, y8=y8)
    assert same_form(y8, quantized(sign * w.double(), f8)[0])


def test_what_a_gate_is_does_not_hang_on_the_rows():
    """Micro-batches of which one has a single row: the gradient of one number is gathered over all of them; a
    token's is written."""
    cols, w = 300, torch.ones(300, device="cuda")
    gate, total, each = torch.full((1,), 0.5, device="cuda"), torch.zeros(1, device="cuda"), []
    for rows in (3, 1, 2):
        o, h, dy = (torch.randn(rows, cols, device="cuda", generator=gen(rows + i)).to(BF16) for i in (10, 20, 30))
        ws = torch.empty(zs.zero_gated_norms_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        args = (dy, o, h, w, torch.ones(rows, device="cuda"), torch.empty_like(o), torch.empty_like(o), ws)
        zs.zero_gated_norms_backward(*args, gate=gate, dgate=total, add=True)
        each.append(torch.zeros(1, device="cuda"))
        zs.zero_gated_norms_backward(*args, gate=gate, dgate=each[-1])
        token = torch.full((rows, 1), 7.0, device="cuda")
        zs.zero_gated_norms_backward(*args, gate=gate.expand(rows, 1).contiguous(), dgate=token, add=True)
        written = torch.zeros(rows, 1, device="cuda")
        zs.zero_gated_norms_backward(*args, gate=gate.expand(rows, 1).contiguous(), dgate=written)
        assert torch.equal(token, written)
        if rows > 1:
            with pytest.raises(ValueError):
                zs.zero_gated_norms_backward(*args, gate=gate.view(1, 1), dgate=total.view(1, 1), add=True)
    assert torch.equal(total, each[0] + each[1] + each[2])
    assert zs.layer._gate_kind(gate.view(1, 1), 1, cols) == zs.layer.GATE_ROWS


@pytest.mark.parametrize("f8", [E4M3, E5M2])
def test_restored_blocks_that_are_infinite(f8):
    """A transposed block with an infinite scale has zeros for its numbers, as zero_fp8_quantize's has."""
    q = whole(1, (200, 130), -15, 15).to(f8)
    s = torch.ones(2, 200, device="cuda")
    col = torch.ones(130, device="cuda")
    col[5], col[129] = float("inf"), float("inf")
    q[:, [5, 129]] = torch.ones(200, 2, device="cuda").to(f8)
    got, want, x = pair(130, 200, f8), pair(130, 200, f8), torch.empty(200, 130, device="cuda")
    zs.zero_fp8_restore(q, s, col=col, x=x, t8=got)
    zs.zero_fp8_quantize(x.t().contiguous(), *want)
    assert x[:, 5].isinf().all() and same_form(got, want)


# widths that fill the lanes of every kernel, and widths that leave some of them, or a part of a unit, empty
FILLED = [1, 100, 128, 250, 256, 1000, 1001, 1024, 2300, 2304, 2560, 4000, 4096, 4100, 8192, 9000, 16384, 16390, 16392, 20000]


@pytest.mark.parametrize("cols", FILLED)
@pytest.mark.parametrize("kind", ["one", "rows"])
def test_an_infinite_gate_at_every_width(cols, kind):
    """h is infinite, so its squares' sum is and rstd_pre = 0, and so is each block's scale."""
    rows, inf = 5, float("inf")
    for pad in (0, 8 - cols % 8):
        o = strided((torch.randint(0, 2, (rows, cols), device="cuda", generator=gen(1)) * 2 - 1).to(BF16), pad, float("nan"))
        x = strided(torch.ones(rows, cols, device="cuda", dtype=BF16), pad, float("nan"))
        gate = torch.full((rows, 1) if kind == "rows" else (1,), inf, device="cuda")
        hit = torch.ones(rows, dtype=torch.bool, device="cuda")
        if kind == "rows":
            gate[2:] = 0.5
            hit[2:] = False
        h, h8, y8, rstd = torch.empty_like(o), pair(rows, cols), pair(rows, cols), torch.full((rows,), 7.0, device="cuda")
        w = torch.ones(cols, device="cuda")
        for w_post in (None, w):
            zs.zero_gated_norms_fp8(o, x, w, 1e-5, h, w_post=w_post, gate=gate, y8=y8, h8=h8, rstd_pre=rstd)
            assert (rstd[hit] == 0).all() and h[hit].isinf().all() and (h8[1][:, hit] == inf).all()
            assert y8[1][:, hit].isnan().all()  # infinity times 0
            assert rstd[~hit].isfinite().all() and (rstd[~hit] > 0).all() and h8[1][:, ~hit].isfinite().all()


@pytest.mark.parametrize("cols", FILLED)
def test_rows_whose_squares_vanish_at_every_width(cols):
    """eps = 0 and squares below fp32's smallest: rstd is infinite, and so is each element of y and each scale."""
    x = strided(torch.full((3, cols), 2.0 ** -100, device="cuda", dtype=BF16), 8 - cols % 8, float("nan"))
    y8, rstd = pair(3, cols), torch.empty(3, device="cuda")
    zs.zero_gated_norms_fp8(torch.zeros_like(x), x, torch.ones(cols, device="cuda"), 0.0, torch.empty_like(x), y8=y8, rstd_pre=rstd)
    assert rstd.isinf().all() and (y8[1] == float("inf")).all()


@pytest.mark.parametrize("cols", [1, 7, 100, 128, 131, 250, 1000, 1003])
@pytest.mark.parametrize("pad", [0, 16])
def test_gradients_of_an_infinite_block_at_every_width(cols, pad):
    """v's last block is infinite: du8's scale of it is too, and dv8 is as without it."""
    rows, kb = 133, (cols + 127) // 128
    da, u, v = (torch.full((rows, cols), c, device="cuda") for c in (0.5, 40.0, -2.0))
    u, v = (strided(t.to(E4M3), pad + 16 - cols % 16 if pad else 0, 5.0) for t in (u, v))
    su, sv = torch.ones(kb, rows, device="cuda"), torch.ones(kb, rows, device="cuda")
    sv[-1, ::2] = float("inf")
    out = dict(du8=pair(rows, cols), dv8=pair(rows, cols), du8t=pair(cols, rows), dv8t=pair(cols, rows), a8t=pair(cols, rows))
    zs.zero_activation_backward_fp8(da.to(BF16), u, v, "silu", su=su, sv=sv, **out)
    assert (out["du8"][1][-1, ::2] == float("inf")).all() and out["du8"][1][:, 1::2].isfinite().all()
    assert out["du8"][1][:-1].isfinite().all() and (out["dv8"][1] == 20.0 / torch.tensor(448.0)).all()
    last = (cols - 1) // 128 * 128
    for k in ("du8t", "a8t"):
        assert (out[k][1][:, last:] == float("inf")).all() and out[k][1][:, :last].isfinite().all()
    assert same_form(out["dv8t"], quantized(torch.full((cols, rows), 20.0, device="cuda", dtype=torch.float64), E4M3)[0])


@pytest.mark.parametrize("cols", [100, 200, 1000, 2300, 4000, 8000, 9000])
@pytest.mark.parametrize("kind", ["none", "one", "cols", "rows"])
@pytest.mark.parametrize("s8", [True, False])
def test_gradients_without_a_norm_behind_do_not_read_o(cols, kind, s8):
    """d_o = gate * dH there: an o that is not finite changes neither d_o nor dx, and dgate alone."""
    a = backward_inputs(19, cols, BF16, F32, kind, False, s8)
    want = run_backward(scale=0.5, **a)
    a["o"][3] = float("nan")
    if s8:
        a["so"][0, 5], a["so"][-1, 7] = float("inf"), float("nan")
    else:
        a["o"][5, 0], a["o"][7, cols - 1] = float("inf"), float("-inf")
    got = run_backward(scale=0.5, **a)
    assert torch.equal(got["d_o"], want["d_o"]) and torch.equal(got["dx"], want["dx"])
    assert torch.equal(got["dw_pre"], want["dw_pre"])
    if kind == "rows":
        bad = torch.tensor([3, 5, 7], device="cuda")
        good = torch.ones(19, dtype=torch.bool, device="cuda").index_fill_(0, bad, False)
        assert not got["dgate"][bad].isfinite().any() and torch.equal(got["dgate"][good], want["dgate"][good])
    elif kind != "none":
        assert not got["dgate"].isfinite().all()


# ----------------------------------------------------------------- calls that the description allows

@pytest.mark.parametrize("rows,cols", [(1, 9), (128, 256), (131, 264), (257, 1001)])
@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("over", ["du", "dv"])
def test_gradients_over_da_with_transposed_forms(rows, cols, s8, over):
    """The columns are formed again behind the rows, which have been written over da by then."""
    args, _ = exact_act(rows, cols, BF16, s8, True, 30)
    da, u, v, su, sv = args

    def run(halves):
        out = dict(du8=pair(rows, cols, E5M2), dv8t=pair(cols, rows, E5M2), du8t=pair(cols, rows, E5M2), a8t=pair(cols, rows))
        zs.zero_activation_backward_fp8(da, u, v, "gelu", su=su, sv=sv, **out, **halves)
        return out

    halves = dict(du=torch.empty_like(da), dv=torch.empty_like(da))
    want = run(halves)
    other = "dv" if over == "du" else "du"
    mine = {over: da, other: torch.empty_like(da)}
    got = run(mine)
    assert all(same_form(got[k], want[k]) for k in want)
    assert torch.equal(mine["du"], halves["du"]) and torch.equal(mine["dv"], halves["dv"])


@pytest.mark.parametrize("cols", [96, 200, 1000, 2304, 4096, 8192, 8200])
@pytest.mark.parametrize("crossed", [False, True])
def test_norms_backward_of_halves_in_place(cols, crossed):
    a = backward_inputs(50, cols, BF16, F32, "rows", True, False)
    want = run_backward(scale=1.0, **a)
    dgate = torch.empty_like(want["dgate"])
    d_o, dx = (a["dh"], a["dy"]) if crossed else (a["dy"], a["dh"])
    zs.zero_gated_norms_backward(a["dy"], a["o"], a["h"], a["w_pre"], a["rh"], d_o, dx, None, dh=a["dh"], w_post=a["w_post"],
                                 rstd_post=a["ro"], gate=a["gate"], dgate=dgate)
    assert torch.equal(d_o, want["d_o"]) and torch.equal(dx, want["dx"]) and torch.equal(dgate, want["dgate"])


def test_sums_of_no_rows_behind_other_work_in_a_graph():
    """The columns' kernel is launched early; here it is the call's only one, behind a fill and a copy."""
    a = backward_inputs(0, 200, BF16, F32, "cols", True, True)
    ws = torch.empty(zs.zero_gated_norms_workspace_bytes(0, 200), dtype=torch.uint8, device="cuda")
    z, dw, src = torch.empty(0, 200, device="cuda", dtype=BF16), torch.empty(200, device="cuda"), torch.ones(200, device="cuda")
    other = torch.empty(200, device="cuda")

    def run():
        dw.fill_(3.0)
        zs.zero_gated_norms_backward(a["dy"], a["o"], a["h"], a["w_pre"], a["rh"], z, z.clone(), ws, so=a["so"], sh=a["sh"],
                                     w_post=a["w_post"], rstd_post=a["ro"], gate=a["gate"], dw_pre=dw, add=True)
        other.copy_(dw)
        zs.zero_gated_norms_backward(a["dy"], a["o"], a["h"], a["w_pre"], a["rh"], z, z.clone(), ws, so=a["so"], sh=a["sh"],
                                     w_post=a["w_post"], rstd_post=a["ro"], gate=a["gate"], dw_pre=dw)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    dw.copy_(src)
    other.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert (other == 3.0).all() and (dw == 0).all()


def test_activation_gradients_side_by_side_and_in_graphs():
    """Four streams at once, and the same calls captured and replayed on new inputs: the transposed forms too."""
    rows, cols = 700, 1096
    sets = [exact_act(rows, cols, BF16, True, True, 50 + 10 * i)[0] for i in range(4)]
    outs = [dict(du8=pair(rows, cols), dv8=pair(rows, cols), du8t=pair(cols, rows), dv8t=pair(cols, rows), a8t=pair(cols, rows)) for _ in sets]

    def run(args, out):
        da, u, v, su, sv = args
        zs.zero_activation_backward_fp8(da, u, v, "silu", su=su, sv=sv, **out)

    wants = []
    for args, out in zip(sets, outs):
        run(args, out)
        wants.append({k: (q.clone(), s.clone()) for k, (q, s) in out.items()})
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for st, args, out in zip(streams, sets, outs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                run(args, out)
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert all(same_form(out[k], want[k]) for out, want in zip(outs, wants) for k in want)
    static = tuple(t.clone() for t in sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(static, outs[0])
    for args, want in zip(sets, wants):
        for to, t in zip(static, args):
            to.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_form(outs[0][k], want[k]) for k in want)
