"""The operators around the step where rounding, range, lengths and sharing of
buffers are at their edges."""
import json
import math
import os
import subprocess
import sys

import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from ops_reference import QMAX, TINY, U, blocks, clip_factor, half_ulp, rmsnorm_backward
from test_gpu_ops import (BF16, E4M3, E5M2, F16, F32, backward_case, chain, check_product, gen, normal, operand,
                          workspace)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- 8-bit blocks

def divided(x, f8, tile):
    """x's 8-bit form by fp32 divisions: every bit is determined."""
    r, k = x.shape
    a = torch.zeros(blocks(r) * 128, blocks(k) * 128, device="cuda")
    a[:r, :k] = x.float().abs()
    a = a.view(-1, blocks(k), 128).amax(2)[:r]
    if tile:
        a = torch.nn.functional.pad(a, (0, 0, 0, -r % 128)).view(-1, 128, blocks(k)).amax(1)
    s = (a / torch.full_like(a, QMAX[f8])).clamp_min(TINY)  # (by a number, torch multiplies by its reciprocal)
    at = s.repeat_interleave(128, 1)[:, :k]
    at = at.repeat_interleave(128, 0)[:r] if tile else at
    return (x.float() / at).to(f8), s.t().contiguous()


def same_bits(a, b):
    """Equal as numbers, zeros with their signs, NaNs in the same places."""
    nan = a.float().isnan()
    assert torch.equal(nan, b.float().isnan())
    ba, bb = (t.contiguous().view(torch.uint8) for t in (a, b))
    if a.element_size() == 1:
        assert torch.equal(ba[~nan], bb[~nan])
    else:
        assert torch.equal(a[~nan], b[~nan])


KINDS = {
    "normal": lambda g, n: torch.randn(n, device="cuda", generator=g),
    # few bits: quotients that are the middle between two 8-bit values are common
    "few bits": lambda g, n: torch.randint(-16, 17, n, device="cuda", generator=g) * 0.125,
    "tiny": lambda g, n: torch.randn(n, device="cuda", generator=g) * 2.0 ** -100,
    "subnormal": lambda g, n: torch.randn(n, device="cuda", generator=g) * 2.0 ** -124,
    "huge": lambda g, n: torch.randn(n, device="cuda", generator=g).clamp(-3, 3) * 2.0 ** 126,
    "spread": lambda g, n: torch.exp2(torch.rand(n, device="cuda", generator=g) * 60 - 40),
}


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype,f8", [(BF16, E4M3), (F16, E4M3), (F32, E4M3), (BF16, E5M2), (F16, E5M2), (F32, E5M2)])
@pytest.mark.parametrize("kind", KINDS)
def test_quantize_rounds_the_quotient(kind, dtype, f8, tile):
    x = KINDS[kind](gen(7), (300, 1000))
    x[17, 200:240] = -0.0
    x = x.to(dtype)
    if dtype == F16:
        x[x.isinf()] = 1.0
    q, s = zs.fp8_empty(300, 1000, f8, tile)
    qt, st = zs.fp8_empty(1000, 300, f8, tile)
    zs.zero_fp8_quantize(x, q, s, qt, st, tile=tile)
    for got, got_s, want in ((q, s, divided(x, f8, tile)), (qt, st, divided(x.t(), f8, tile))):
        assert torch.equal(got_s, want[1])
        same_bits(got, want[0])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("tile", [False, True])
def test_quantize_divides_what_is_not_finite(bad, tile):
    x = normal(1, (130, 300), BF16)
    x[3, 140] = bad
    x[3, 141] = -0.0
    q, s = zs.fp8_empty(130, 300, E4M3, tile)
    qt, st = zs.fp8_empty(300, 130, E4M3, tile)
    zs.zero_fp8_quantize(x, q, s, qt, st, tile=tile)
    for got, got_s, want in ((q, s, divided(x, E4M3, tile)), (qt, st, divided(x.t(), E4M3, tile))):
        same_bits(got_s, want[1])
        same_bits(got, want[0])


@pytest.mark.parametrize("wdtype,f8", [(BF16, E4M3), (F16, E5M2), (F32, E4M3)])
@pytest.mark.parametrize("cols", [256, 1024, 2048, 4096, 8192, 16384, 32768])
def test_rmsnorm_rounds_the_quotient(cols, wdtype, f8):
    """Rows whose squares have the mean 4 exactly: rstd is 1/2 and y one product."""
    eight = torch.tensor([[5, 2, 1, 1, 1, 0, 0, 0], [4, 3, 2, 1, 1, 1, 0, 0], [3, 3, 3, 2, 1, 0, 0, 0.]], device="cuda")
    g, rows = gen(3), 6
    pick = torch.randint(0, 3, (rows, cols // 8), device="cuda", generator=g)
    sign = torch.randint(0, 2, (rows, cols), device="cuda", generator=g) * 2.0 - 1.0
    x = (eight[pick].view(rows, cols) * sign).to(BF16)
    w = (1 + normal(2, (cols,), F32, 0.2)).to(wdtype)
    q, s = zs.fp8_empty(rows, cols, f8)
    rstd = torch.empty(rows, device="cuda")
    zs.zero_rmsnorm_fp8(x, w, 0.0, rstd, q=q, s=s)
    assert (rstd == 0.5).all()
    want, want_s = divided(x.float() * 0.5 * w.float(), f8, False)
    assert torch.equal(s, want_s)
    same_bits(q, want)


# ----------------------------------------------------------------- clip

def clipped(xs, outs, inv, max_norm, stat):
    """zero_tensors_clip against the formula in 64 bits: the factor's rounding, the product's, out's."""
    sumsq = zs.read_tensors_stat(stat).sumsq
    before = [x.double() for x in xs]
    zs.zero_tensors_clip(xs, outs, inv, max_norm, stat)
    for x, o in zip(before, xs if outs is None else outs):
        want = x * clip_factor(sumsq, inv, max_norm)
        assert ((o.double() - want).abs() <= want.abs() * 6 * U + half_ulp(want, o.dtype) * (1 + 1e-6)).all()


def norm_of(xs, inv):
    ws = torch.zeros(zs.zero_tensors_workspace_bytes(xs), dtype=torch.uint8, device="cuda")
    stat = zs.new_tensors_stat()
    zs.zero_tensors_norm(xs, inv, stat, ws)
    return stat


@pytest.mark.parametrize("out", [None, F32, BF16])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e30])
@pytest.mark.parametrize("inv", [1.0, 2.0 ** -4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_clip_where_the_norm_leaves_fp32(dtype, inv, max_norm, out):
    """Finite gradients whose norm is 2^128 or more: clipped, not zeroed."""
    xs = [normal(1, (20_011,), F32).clamp(-3, 3).mul_(1e38).to(dtype), normal(2, (333,), F32).mul_(1e37).to(dtype),
          normal(3, (5,), BF16)]
    stat = norm_of(xs, inv)
    got = zs.read_tensors_stat(stat)
    assert got.found_inf == 0 and got.sumsq > 2.0 ** 256
    clipped(xs, None if out is None else [torch.empty(x.shape, dtype=out, device="cuda") for x in xs], inv, max_norm, stat)


def test_clip_of_two_elements_near_the_largest():
    x = torch.tensor([3e38, -3e38], device="cuda")
    stat = norm_of([x], 1.0)
    clipped([x], None, 1.0, 1.0, stat)
    assert torch.allclose(x, torch.tensor([0.5 ** 0.5, -0.5 ** 0.5], device="cuda"), rtol=1e-6)


@pytest.mark.parametrize("inv", [2.0 ** -110, 2.0 ** -30, 1.0])
@pytest.mark.parametrize("sumsq", [1e-60, 1e-30, 1e60, 1e90])
def test_clip_with_a_sum_from_elsewhere(sumsq, inv):
    """The sum over ranks is the caller's, anywhere in binary64's range."""
    x = normal(4, (5000,), F32, 1e35 if inv < 1e-30 or sumsq > 1e59 else 1.0)
    stat = zs.new_tensors_stat()
    stat[:8].view(torch.float64).fill_(sumsq)
    clipped([x], [torch.empty_like(x)], inv, 1.0, stat)


@pytest.mark.parametrize("sumsq", [float("inf"), float("nan")])
def test_clip_leaves_what_has_no_finite_sum(sumsq):
    x = normal(4, (5000,), F32)
    before, stat = x.clone(), zs.new_tensors_stat()
    stat[:8].view(torch.float64).fill_(sumsq)
    zs.zero_tensors_clip([x], None, 1.0, 1.0, stat)
    assert torch.equal(x, before)


@pytest.mark.parametrize("max_norm", [1e-300, 1e-46, 1e-40, 1e-37, 1e37, 1e39, 1e300, float("inf")])
@pytest.mark.parametrize("size", [1e-2, 1e30])
def test_clip_to_limits_outside_fp32(size, max_norm):
    """A positive limit clips, however small; no limit is too large."""
    x = normal(4, (5000,), F32, size)
    before, stat = x.clone(), norm_of([x], 1.0)
    clipped([x], None, 1.0, max_norm, stat)
    assert torch.equal(x, before) == (max_norm > 1e34)


@pytest.mark.parametrize("scale", [1.0, 1024.0, 2.0 ** 16])
def test_norm_clip_and_step_under_a_loss_scale(scale):
    """Gradients of a loss times `scale`: the norm's inv_scale is 1 / scale, the
    clip's is 1, for the step divides what it reads by its state's own scale.
    Elements that fp16 does not hold without the scale reach the moments."""
    sizes, max_norm = [(300, F16), (4097, F16), (64, F32), (1001, F16)], 1e-6
    z = zs.ZeroStep([n for n, _ in sizes], 1, zs.F16, zs.adam_cfg(), loss_scale=scale)
    flat = torch.zeros(z.grad_numel(), dtype=F16, device="cuda")
    outs = [flat[o:o + n] for o, (n, _) in zip(z.offsets, sizes)]
    small = 1e-3 if scale == 1.0 else 1e-8
    xs = [normal(i, (n,), F32, small * scale).to(t) for i, (n, t) in enumerate(sizes)]
    stat = norm_of(xs, 1.0 / scale)
    zs.zero_tensors_clip(xs, outs, 1.0, max_norm, stat)
    z.step([flat])
    st = z.read_state()
    assert (st.t, st.skipped) == (1, 0)
    # (1e-6 beside the norm is part of the factor)
    c = clip_factor(sum(float((x.double() / scale).square().sum()) for x in xs), 1.0, max_norm)
    assert c < 0.9
    for x, o, n in zip(xs, z.offsets, (n for n, _ in sizes)):
        m, kept = z.m[st.cur][o:o + n].double(), x.double() * c
        want = kept / scale * 0.1
        assert ((m - want).abs() <= want.abs() * 16 * U + half_ulp(kept, F16) * (1 + 1e-6) * 0.1 / scale).all()
        assert scale == 1.0 or (m != 0).double().mean() > 0.95
    xs[1][5] = float("inf")
    stat = norm_of(xs, 1.0 / scale)
    zs.zero_tensors_clip(xs, outs, 1.0, max_norm, stat)
    z.step([flat])
    assert (z.read_state().t, z.read_state().skipped) == (1, 1)


# ----------------------------------------------------------------- product

def test_matmul_whose_waits_run_out_reports_and_leaves_the_workspace_ready():
    """With ZERO_TEST_MATMUL_GIVE_UP=1 (read once per process: a child) every
    second CTA takes a wait that its first poll does not end as run out: the
    error word is set and every tile's counter is back at zero."""
    env = dict(os.environ, ZERO_TEST_MATMUL_GIVE_UP="1")
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "gpu_ops_children.py"), "give_up"], capture_output=True,
                       text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert json.loads(r.stdout.strip().splitlines()[-1]) == {"ok": True}


def test_example_stops_on_a_product_that_gave_up():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from fp8_layer import Layer, train
    layer = Layer(128, 128, 256)
    x, residual, target = (normal(i, (128, 128), BF16) for i in range(3))
    train(layer, x, residual, target, 1)
    layer.mm_ws[0] = 1
    with pytest.raises(RuntimeError):
        train(layer, x, residual, target, 1)


@pytest.mark.parametrize("tile,add", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("n,k", [(40_000, 129), (50_257, 769), (39_000, 1100)])
@pytest.mark.parametrize("m", [1, 17, 64])
def test_matmul_of_few_rows_walks_many_columns(m, n, k, tile, add):
    """More tiles than two to an SM: a CTA takes several, its rings of stages, sums and scales in the middle of a turn."""
    a, sa = operand(m, m, k, E4M3, False)
    b, sb = operand(n, n, k, E5M2 if add else E4M3, tile)
    out = normal(3, (m, n), F32 if add else BF16, 5.0)
    before, ws = out.double(), workspace(m, n, k)
    zs.zero_fp8_matmul(a, sa, b, sb, out, ws, add=add)
    check_product(out, a, sa, b, sb, before if add else None)
    assert not zs.read_matmul_error(ws)


# ----------------------------------------------------------------- norm and clip over lists

@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("sizes,at", [([9000] * 1100, 0), ([9000] * 1100, 1099), ([3_000_001] * 5, 4), ([50_000] * 2300, 3)])
def test_norm_of_a_long_list_finds_what_is_not_finite(sizes, at, bad):
    """Lists whose norm ends in a kernel of its own, and several launches to a list."""
    dtype = (BF16, F32)[at % 2]
    xs = [normal(i, (n,), dtype) for i, n in enumerate(sizes)]
    ws = torch.zeros(zs.zero_tensors_workspace_bytes(xs), dtype=torch.uint8, device="cuda")
    each = torch.empty(len(xs), dtype=torch.float64, device="cuda")
    xs[at][-1] = bad
    stat = zs.new_tensors_stat()
    zs.zero_tensors_norm(xs, 1.0, stat, ws, each)
    got = zs.read_tensors_stat(stat)
    assert got.found_inf == 1 and not math.isfinite(got.sumsq) and not math.isfinite(got.norm)
    ok = torch.ones(len(xs), dtype=torch.bool)
    ok[at] = False
    assert each[ok.cuda()].isfinite().all() and not math.isfinite(float(each[at]))
    zs.zero_tensors_clip(xs, None, 1.0, 1e-3, stat)  # nothing is clipped
    assert torch.equal(xs[0][:100], normal(0, (sizes[0],), dtype)[:100])
    xs[at][-1] = 0.0
    zs.zero_tensors_norm(xs, 1.0, stat, ws)  # and the workspace carries nothing over
    assert zs.read_tensors_stat(stat).found_inf == 0
    assert int(ws[:8].sum()) == 0


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_clip_with_a_factor_of_one_keeps_every_bit(dtype):
    """Every half value (fp32: 2^21 patterns over the whole range) but NaNs, in place and copied."""
    if dtype == F32:
        x = torch.arange(0, 1 << 32, 2047, device="cuda").to(torch.int32).view(F32)
    else:
        x = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[torch.isfinite(x)].contiguous()
    word = torch.int32 if dtype == F32 else torch.int16
    before, y, stat = x.clone(), torch.empty_like(x), zs.new_tensors_stat()
    for max_norm in (0.0, 1e30):  # no limit, and one above the stat's norm of 0
        zs.zero_tensors_clip([x], [y], 1.0, max_norm, stat)
        zs.zero_tensors_clip([x], None, 1.0, max_norm, stat)
        assert torch.equal(x.view(word), before.view(word)) and torch.equal(y.view(word), before.view(word))


# ----------------------------------------------------------------- root-mean-square norm

@pytest.mark.parametrize("cols", [257, 1001, 4096, 9001, 17000, 17008])
def test_rmsnorm_sum_over_the_residual(cols):
    x, r, w = normal(1, (9, cols), BF16), normal(2, (9, cols), BF16), normal(3, (cols,), F32)
    h, y, y2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    (q, s), (q2, s2) = zs.fp8_empty(9, cols), zs.fp8_empty(9, cols)
    zs.zero_rmsnorm_fp8(x, w, 1e-5, residual=r, h=h, y=y, q=q, s=s)
    zs.zero_rmsnorm_fp8(x, w, 1e-5, residual=r, h=r, y=y2, q=q2, s=s2)
    assert torch.equal(r, h) and torch.equal(y2, y) and torch.equal(s2, s)
    same_bits(q2, q)


@pytest.mark.parametrize("dtype,dwt", [(BF16, F32), (F16, F16)])
@pytest.mark.parametrize("rows,cols", [(10_001, 200), (2500, 1000), (1300, 2048), (1000, 4096), (611, 4095), (400, 8192),
                                       (400, 9001), (333, 12_288), (200, 16_384)])
def test_rmsnorm_backward_of_many_rows(rows, cols, dtype, dwt):
    """More rows than CTAs: the next row on its way while this one is reduced,
    sums of dw over a CTA's rows, outputs over inputs that later rows still read."""
    h, dy, w, dr, rstd = backward_case(rows, cols, dtype, True, seed=rows)
    dx, dw = torch.empty_like(h), torch.empty(cols, dtype=dwt, device="cuda")
    nbytes = zs.zero_rmsnorm_workspace_bytes(rows, cols)
    parts = nbytes // (4 * cols)
    assert parts < rows
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda").fill_(255)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dr)
    want, want_w, size, size_w = rmsnorm_backward(dy.double(), h.double(), w.double(), rstd.double(), dr.double())
    tol = size * (chain(cols) + 4) * U
    assert ((dx.double() - want).abs() <= tol + half_ulp(want, dtype) * (1 + 1e-6)).all()
    # xhat's rounding, a CTA's rows, the CTAs' sums by 32 or 128 threads, two shuffles, 8 or 32 warps
    steps = 1 + -(-rows // parts) + -(-parts // (128 if parts > 512 else 32)) + 2 + (32 if parts > 512 else 8)
    tol_w = size_w * steps * U
    assert ((dw.double() - want_w).abs() <= tol_w + half_ulp(want_w, dwt) * (1 + 1e-6)).all()
    before = normal(9, (cols,), dwt)
    added = before.clone()
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, added, ws, dres=dr, add_dw=True)
    sum_w = want_w + before.double()
    assert ((added.double() - sum_w).abs() <= tol_w + sum_w.abs() * U + half_ulp(sum_w, dwt) * (1 + 1e-6)).all()
    for over in (dy.clone(), dr.clone()):
        on_dy = torch.equal(over, dy)
        again = torch.empty_like(dw)
        zs.zero_rmsnorm_backward(over if on_dy else dy, h, w, rstd, over, again, ws, dres=dr if on_dy else over)
        assert torch.equal(over, dx) and torch.equal(again, dw)
    alone = torch.empty_like(dx)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, alone, None, None, dres=dr)  # without dw
    assert torch.equal(alone, dx)
