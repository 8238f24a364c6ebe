"""The operators around the step against plain 64-bit forms on the GPU.

Tolerances follow from the formats: u = 2^-24 is an fp32 operation's relative
error, a sum of n terms in any order is off by at most (n - 1) u times the sum
of their magnitudes, and a stored result by half a unit in the last place of
its type."""
import math

import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from ops_reference import (QMAX, U, at_elements, blocks, clip_factor, half_ulp, matmul, rmsnorm,
                           rmsnorm_backward, scales)

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, shape, dtype=F32, sigma=1.0):
    return (torch.randn(shape, device="cuda", generator=gen(seed)) * sigma).to(dtype)


def strided(x, pad, fill):
    """x as a view whose rows are `pad` elements further apart, the gaps filled."""
    if pad == 0:
        return x
    big = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=F32, device="cuda").to(x.dtype)
    big[:, :x.shape[1]] = x
    return big[:, :x.shape[1]]


def gap(view):
    """What lies between a strided view's rows."""
    base = view._base
    return base[:, view.shape[1]:].float() if base is not None else torch.zeros(0)


# ----------------------------------------------------------------- norm and clip

def norm_of(tensors, inv=1.0, per=False):
    ws = torch.zeros(zs.zero_tensors_workspace_bytes(tensors), dtype=torch.uint8, device="cuda")
    stat = zs.new_tensors_stat()
    each = torch.full((len(tensors),), -1.0, dtype=torch.float64, device="cuda") if per else None
    zs.zero_tensors_norm(tensors, inv, stat, ws, each)
    again = zs.new_tensors_stat()
    zs.zero_tensors_norm(tensors, inv, again, ws)
    assert torch.equal(stat, again)               # the workspace is ready for the next call
    assert int(ws[:8].sum()) == 0
    return stat, each


LISTS = {
    "none": [],
    "empty": [(0, BF16), (0, F32)],
    "one": [(1, F16)],
    "odd": [(7, BF16), (0, F16), (4096, F16), (4097, F32), (1, F32), (12289, BF16)],
    "many": [((37 * i) % 1009, (F16, BF16, F32)[i % 3]) for i in range(2100)],
    "long": [(30_000_001, BF16), (5, F32), (9_000_000, F16), (1_000_003, F32)],
}


@pytest.mark.parametrize("inv", [1.0, 2.0 ** -10])
@pytest.mark.parametrize("name", LISTS)
def test_norm_over_many_tensors(name, inv):
    xs = [normal(i, (n,), t, 0.5) for i, (n, t) in enumerate(LISTS[name])]
    stat, each = norm_of(xs, inv, per=True)
    got = zs.read_tensors_stat(stat)
    want = [float((x.double() * inv).square().sum()) for x in xs]
    total = math.fsum(want)
    # a thread's running sums take chunk / 2048 squares, then pairs of values
    chunk = max(4096, sum(x.numel() for x in xs) // 16384 + 4096)
    tol = (chunk / 2048 + 4) * U
    assert abs(got.sumsq - total) <= tol * total
    assert abs(got.norm - math.sqrt(total)) <= (tol + U) * math.sqrt(total)
    assert got.found_inf == 0
    for a, b in zip(each.tolist(), want):
        assert abs(a - b) <= tol * b


@pytest.mark.parametrize("dtype,big", [(BF16, 1e30), (F32, 1e30), (F32, 1e-30), (BF16, 1e-36), (F32, 0.0)])
def test_norm_of_values_whose_squares_leave_fp32(dtype, big):
    x = normal(3, (10_001,), F32).mul_(big).to(dtype)
    stat, _ = norm_of([x, torch.zeros(50_000, device="cuda")])
    got = zs.read_tensors_stat(stat)
    want = float(x.double().square().sum())
    assert abs(got.sumsq - want) <= 1e-6 * want and got.found_inf == 0
    assert abs(got.norm - math.sqrt(want)) <= 1e-6 * math.sqrt(want)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_norm_finds_what_is_not_finite(bad, dtype):
    xs = [normal(1, (5000,), dtype), normal(2, (9000,), dtype)]
    xs[1][8999] = bad
    stat, _ = norm_of(xs)
    got = zs.read_tensors_stat(stat)
    assert got.found_inf == 1 and not math.isfinite(got.sumsq)
    # nothing is clipped: the gradients reach the step with what is not finite
    out = [torch.empty_like(x) for x in xs]
    zs.zero_tensors_clip(xs, out, 1.0, 0.01, stat)
    for a, b in zip(out, xs):  # a product keeps no NaN's payload
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])
    ys = [normal(1, (5000,), dtype)]
    ok, _ = norm_of(ys)
    assert zs.read_tensors_stat(ok).found_inf == 0


@pytest.mark.parametrize("sizes", [[9000] * 1100, [3_000_001] * 5, [7] * 600, [50_000, 40_000]])
def test_norm_and_clip_in_a_row(sizes):
    """In place, each norm's reader and the next norm's writer back to back, short lists and long ones."""
    xs = zs.tensor_list([normal(i, (n,), F32) for i, n in enumerate(sizes)])
    ws = torch.zeros(zs.zero_tensors_workspace_bytes(xs), dtype=torch.uint8, device="cuda")
    limits = [16.0, 8.0, 2.0, 0.5, 0.25]
    stats = [zs.new_tensors_stat() for _ in limits + [0]]
    for stat, limit in zip(stats, limits):
        zs.zero_tensors_norm(xs, 1.0, stat, ws)
        zs.zero_tensors_clip(xs, None, 1.0, limit, stat)
    zs.zero_tensors_norm(xs, 1.0, stats[-1], ws)
    for stat, limit in zip(stats[1:], limits):
        # the 1e-6 beside a norm of 0.5 or more, the factor's and the elements' roundings, the norm's own
        assert abs(zs.read_tensors_stat(stat).norm - limit) <= limit * (2e-6 + 24 * U)


@pytest.mark.parametrize("max_norm", [0.0, 0.25, 1e9])
@pytest.mark.parametrize("out_dtype", [F16, BF16, F32, None])
def test_clip(max_norm, out_dtype):
    sizes = [(3, F32), (0, F16), (65_537, BF16), (4096, F16), (129, BF16), (1, F16)]
    inv = 2.0 ** -5
    xs = [normal(i, (n,), t, 3.0) for i, (n, t) in enumerate(sizes)]
    before = [x.clone() for x in xs]
    stat, _ = norm_of(xs, inv)
    f = clip_factor(zs.read_tensors_stat(stat).sumsq, inv, max_norm)
    if out_dtype is None:
        zs.zero_tensors_clip(xs, None, inv, max_norm, stat)
        outs = xs
    else:
        outs = [torch.empty(n, dtype=out_dtype, device="cuda") for n, _ in sizes]
        zs.zero_tensors_clip(zs.tensor_list(xs), zs.tensor_list(outs), inv, max_norm, stat)
    for x, o in zip(before, outs):
        want = x.double() * f
        # the factor: a root, a sum, a quotient and a product; the product with x
        assert ((o.double() - want).abs() <= want.abs() * 6 * U + half_ulp(want, o.dtype) * (1 + 1e-6)).all()


def test_clip_in_place_with_a_factor_of_one_changes_no_bit():
    x = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16)
    x = x[torch.isfinite(x)].contiguous()
    stat = zs.new_tensors_stat()
    zs.zero_tensors_clip([x], None, 1.0, 0.0, stat)
    y = torch.empty_like(x)
    zs.zero_tensors_clip([x], [y], 1.0, 0.0, stat)
    assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("shift_in,shift_out", [(1, 0), (0, 1), (3, 5)])
def test_norm_and_clip_of_unaligned_tensors(shift_in, shift_out):
    n = 20_011
    x = normal(5, (n + 8,), BF16)[shift_in:shift_in + n]
    flat = torch.full((n + 16,), 7.0, dtype=F16, device="cuda")
    o = flat[shift_out:shift_out + n]
    stat, _ = norm_of([x])
    total = float(x.double().square().sum())
    assert abs(zs.read_tensors_stat(stat).sumsq - total) <= 16 * U * total
    zs.zero_tensors_clip([x], [o], 1.0, 1.0, stat)
    want = x.double() * clip_factor(total, 1.0, 1.0)
    assert ((o.double() - want).abs() <= want.abs() * 16 * U + half_ulp(want, F16) * (1 + 1e-6)).all()
    assert (flat[:shift_out] == 7).all() and (flat[shift_out + n:] == 7).all()


# ----------------------------------------------------------------- 8-bit blocks

def check_blocks(x64, q, s, tile, extra=0.0, s_tol=0.0):
    """q and s are x64's 8-bit form; extra: x64's own relative error before the cast."""
    want = scales(x64, q.dtype, tile)
    assert s.shape == want.shape
    assert ((s.double() - want).abs() <= want * (s_tol + U)).all()
    spread = at_elements(s, *x64.shape, tile)
    y = x64 / spread                                  # what is rounded, within 2 u and `extra`
    err = (q.double() - y).abs()
    assert (err <= half_ulp(y, q.dtype) * (1 + 1e-6) + y.abs() * (3 * U + extra)).all()


SHAPES = [(1, 1), (1, 128), (3, 7), (127, 129), (128, 128), (130, 255), (257, 1000), (1000, 16), (5, 4104)]


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype,f8", [(BF16, E4M3), (F16, E4M3), (F32, E5M2), (BF16, E5M2)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype, f8, tile):
    x = normal(rows * 7 + cols, (rows, cols), dtype)
    x[rows // 2] *= 30.0
    x[0, 0] = 0.0
    q, s = zs.fp8_empty(rows, cols, f8, tile)
    qt, st = zs.fp8_empty(cols, rows, f8, tile)
    zs.zero_fp8_quantize(x, q, s, qt, st, tile=tile)
    check_blocks(x.double(), q, s, tile)
    check_blocks(x.double().t(), qt, st, tile)
    if tile:
        assert torch.equal(q.float().t(), qt.float()) and torch.equal(s.t(), st)
    for one in ((q, s, None, None), (None, None, qt, st)):  # each form alone gives the same bits
        other = [torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda") if t is not None
                 else None for t in one]
        zs.zero_fp8_quantize(x, *other, tile=tile)
        for a, b in zip(one, other):
            if a is not None:
                assert torch.equal(a.float(), b.float())


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("pad_in,pad_out", [(1, 3), (8, 16), (5, 8)])
def test_quantize_strides_leave_the_gaps(pad_in, pad_out, tile):
    x = strided(normal(11, (131, 200), BF16), pad_in, float("nan"))
    q = strided(torch.zeros(131, 200, device="cuda").to(E4M3), pad_out, 5.0)
    qt = strided(torch.zeros(200, 131, device="cuda").to(E4M3), pad_out, 5.0)
    s = strided(torch.zeros(2, 2 if tile else 131, device="cuda"), pad_out, 5.0)
    st = strided(torch.zeros(2, 2 if tile else 200, device="cuda"), pad_out, 5.0)
    zs.zero_fp8_quantize(x, q, s, qt, st, tile=tile)
    check_blocks(x.double(), q, s, tile)
    check_blocks(x.double().t(), qt, st, tile)
    for t in (q, qt, s, st):
        assert (gap(t) == 5.0).all()


@pytest.mark.parametrize("f8", [E4M3, E5M2])
def test_quantize_extremes(f8):
    x = torch.zeros(4, 256, device="cuda")
    x[1, :128] = torch.linspace(-1, 1, 128, device="cuda") * 3e38   # near the largest fp32
    x[2, :128] = 1e-44                                              # below the smallest scale
    x[3, 5] = -2.0
    q, s = zs.fp8_empty(4, 256, f8)
    zs.zero_fp8_quantize(x, q, s)
    check_blocks(x.double(), q, s, False)
    assert (q[0].float() == 0).all() and (s[:, 0] == 2.0 ** -126).all()
    assert float(q[3, 5]) == -QMAX[f8]


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("tile", [False, True])
def test_quantize_passes_on_what_is_not_finite(bad, tile):
    x = normal(1, (130, 300), BF16)
    x[3, 140] = bad
    q, s = zs.fp8_empty(130, 300, E4M3, tile)
    qt, st = zs.fp8_empty(300, 130, E4M3, tile)
    zs.zero_fp8_quantize(x, q, s, qt, st, tile=tile)
    v = q.double() * at_elements(s, 130, 300, tile)
    vt = (qt.double() * at_elements(st, 300, 130, tile)).t()
    for got, rows, cols in ((v, slice(0, 128) if tile else slice(3, 4), slice(128, 256)),
                            (vt, slice(0, 128), slice(128, 256) if tile else slice(140, 141))):
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[rows, cols] = True
        assert got[hit].isnan().all() and got[~hit].isfinite().all()


# ----------------------------------------------------------------- product

def operand(seed, rows, k, f8, tile):
    q, s = zs.fp8_empty(rows, k, f8, tile)
    q.copy_(normal(seed, (rows, k), F32, QMAX[f8] / 4).clamp_(-QMAX[f8], QMAX[f8]).to(f8))
    s.copy_(torch.exp(normal(seed + 1, tuple(s.shape))) * (1.0 / QMAX[f8]))
    return q, s


def workspace(m, n, k):
    return torch.zeros(zs.zero_fp8_matmul_workspace_bytes(m, n, k), dtype=torch.uint8, device="cuda")


def check_product(out, a, sa, b, sb, before=None):
    """Within a block the tensor cores' sums may drop bits below 2^-23 of the
    running sum at each of 128 terms; a scale's product, its use and the sum
    over blocks round in fp32."""
    want, size = matmul(a, sa, b, sb)
    k = a.shape[1]
    tol = (2 * min(128, k) + 2 * blocks(k) + 8) * U * size
    if before is not None:
        want = want + before
        tol = tol + want.abs() * U
    assert ((out.double() - want).abs() <= tol + half_ulp(want, out.dtype) * (1 + 1e-6)).all()


SIZES = [(1, 1, 1), (1, 8, 16), (1, 4096, 1024), (2, 129, 127), (16, 256, 128), (17, 1000, 129), (64, 384, 2048),
         (100, 257, 333), (128, 128, 128), (129, 255, 640), (255, 1, 300), (256, 512, 1024), (300, 1031, 769),
         (1, 7, 20000), (513, 640, 4096), (2304, 2500, 300), (4097, 1290, 257), (2560, 2560, 1024), (1025, 2500, 300), (2304, 1290, 257),
         (3001, 2567, 300), (4096, 2304, 640)]


@pytest.mark.parametrize("tile", [True, False])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul(m, n, k, tile):
    ta, tb, to = [(E4M3, E4M3, BF16), (E5M2, E4M3, F32), (E4M3, E5M2, F16), (E5M2, E5M2, BF16)][(m + n) % 4]
    a, sa = operand(m, m, k, ta, False)
    b, sb = operand(n + 100, n, k, tb, tile)
    out = torch.full((m, n), float("nan"), dtype=to, device="cuda")
    ws = workspace(m, n, k)
    zs.zero_fp8_matmul(a, sa, b, sb, out, ws)
    check_product(out, a, sa, b, sb)
    again = torch.empty_like(out)
    zs.zero_fp8_matmul(a, sa, b, sb, again, ws)
    assert torch.equal(out, again)                 # the same bits from the same workspace
    assert int(ws[:4].sum()) == 0                  # no wait ran out


@pytest.mark.parametrize("to", [F16, BF16, F32])
@pytest.mark.parametrize("m,n,k", [(3, 5, 7), (100, 300, 200), (256, 256, 512), (9, 640, 4000), (2400, 2504, 256),
                                   (1300, 2504, 256)])
def test_matmul_adds(m, n, k, to):
    a, sa = operand(1, m, k, E5M2, False)
    b, sb = operand(2, n, k, E4M3, False)
    out = normal(3, (m, n), to, 5.0)
    before = out.double()
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(m, n, k), add=True)
    check_product(out, a, sa, b, sb, before)


@pytest.mark.parametrize("to", [F16, F32])
@pytest.mark.parametrize("pad", [1, 2, 3, 5, 16])
@pytest.mark.parametrize("m,n,k", [(50, 259, 200), (130, 259, 200), (2561, 2323, 130),
                                   (1281, 2323, 130)])
def test_matmul_output_strides_leave_the_gaps(m, n, k, pad, to):
    a, sa = operand(1, m, k, E4M3, False)
    b, sb = operand(2, n, k, E4M3, m > 1000)
    out = strided(torch.zeros(m, n, device="cuda", dtype=to), pad, 5.0)
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(m, n, k))
    check_product(out, a, sa, b, sb)
    assert (gap(out) == 5.0).all()


@pytest.mark.parametrize("shift", [1, 2, 3, 7])
def test_matmul_into_an_unaligned_output(shift):
    m, n, k = 200, 300, 300
    a, sa = operand(1, m, k, E4M3, False)
    b, sb = operand(2, n, k, E4M3, True)
    flat = torch.full((m * n + 16,), 5.0, dtype=BF16, device="cuda")
    out = flat[shift:shift + m * n].view(m, n)
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(m, n, k))
    check_product(out, a, sa, b, sb)
    assert (flat[:shift] == 5).all() and (flat[shift + m * n:] == 5).all()


def test_matmul_of_sizes_that_change_the_kernel():
    """Each side of the rules on the rows and on the number of tiles."""
    for m, n, k, tile in [(15, 700, 1000, True), (16, 700, 1000, False), (17, 700, 1000, True), (32, 130, 5000, False),
                          (33, 130, 5000, True), (64, 513, 2000, False), (65, 513, 2000, True), (256, 19 * 256, 200, True),
                          (256, 19 * 256 + 1, 200, False), (1024, 19 * 256, 200, False), (1025, 19 * 256, 200, True),
                          (1024, 9 * 256, 200, True), (1024, 10 * 256, 200, True), (2048, 19 * 256, 200, False),
                          (2049, 19 * 256, 200, True)]:
        a, sa = operand(m, m, k, E4M3, False)
        b, sb = operand(n, n, k, E5M2, tile)
        out, ws = torch.empty(m, n, device="cuda"), workspace(m, n, k)
        zs.zero_fp8_matmul(a, sa, b, sb, out, ws)
        check_product(out, a, sa, b, sb)
        assert int(ws[:4].sum()) == 0


def test_matmul_reads_no_padding():
    """NaN codes between the rows' ends and their strides, and strided scales."""
    m, n, k = 70, 140, 200
    a, sa = operand(1, m, k, E4M3, False)
    b, sb = operand(2, n, k, E4M3, False)
    a._base.view(torch.uint8)[:, k:] = 0x7F
    b._base.view(torch.uint8)[:, k:] = 0x7F
    sa, sb = strided(sa, 5, float("nan")), strided(sb, 3, float("nan"))
    out = torch.empty(m, n, device="cuda")
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(m, n, k))
    check_product(out, a, sa, b, sb)


def test_matmul_of_nothing():
    a, sa = zs.fp8_empty(5, 0)
    b, sb = zs.fp8_empty(6, 0)
    out = torch.ones(5, 6, device="cuda")
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(5, 6, 0), add=True)
    assert (out == 1).all()
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(5, 6, 0))
    assert (out == 0).all()
    zs.zero_fp8_matmul(a[:0], sa[:, :0], b, sb, out[:0], workspace(0, 6, 0))


@pytest.mark.parametrize("m", [4, 200])
def test_matmul_passes_on_what_is_not_finite(m):
    n, k = 300, 512
    a, sa = operand(1, m, k, E4M3, False)
    b, sb = operand(2, n, k, E4M3, True)
    sa[1, 2] = float("nan")
    a[3].view(torch.uint8)[130] = 0x7F
    out = torch.zeros(m, n, device="cuda", dtype=BF16)
    zs.zero_fp8_matmul(a, sa, b, sb, out, workspace(m, n, k))
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[2] = bad[3] = True
    assert out[bad].isnan().all() and out[~bad].isfinite().all()


def test_matmul_one_workspace_for_many_sizes():
    sizes = [(1, 4096, 20000), (16, 128, 8192), (513, 640, 256), (1, 7, 20000)]
    ws = max((workspace(*s) for s in sizes), key=torch.Tensor.numel)
    for m, n, k in sizes:
        a, sa = operand(m, m, k, E4M3, False)
        b, sb = operand(n, n, k, E4M3, True)
        out = torch.empty(m, n, device="cuda", dtype=BF16)
        zs.zero_fp8_matmul(a, sa, b, sb, out, ws)
        check_product(out, a, sa, b, sb)


def test_matmul_gradients_against_differences():
    """L = <G, A B^T>: the two products that the backward pass makes of 8-bit
    operands are L's derivatives (L is linear in each operand, so a difference
    of L is exact but for its 64-bit rounding)."""
    m, n, k = 70, 200, 150
    x, w, g = normal(1, (m, k), BF16), normal(2, (n, k), BF16, 0.1), normal(3, (m, n), BF16, 0.01)
    x8, xt8 = zs.fp8_empty(m, k), zs.fp8_empty(k, m)
    w8, wt8 = zs.fp8_empty(n, k, tile=True), zs.fp8_empty(k, n, tile=True)
    g8, gt8 = zs.fp8_empty(m, n, E5M2), zs.fp8_empty(n, m, E5M2)
    zs.zero_fp8_quantize(x, *x8, *xt8)
    zs.zero_fp8_quantize(w, *w8, *wt8, tile=True)
    zs.zero_fp8_quantize(g, *g8, *gt8)

    def value(pair, rows, cols, tile=False):
        return pair[0].double() * at_elements(pair[1], rows, cols, tile)

    dx = torch.empty(m, k, device="cuda")
    dw = torch.zeros(n, k, device="cuda")
    zs.zero_fp8_matmul(*g8, *wt8, dx, workspace(m, k, n))
    zs.zero_fp8_matmul(*gt8, *xt8, dw, workspace(n, k, m), add=True)
    W, G = value(w8, n, k, True), value(g8, m, n)
    v = normal(4, (m, k)).double()
    loss = lambda X: (G * (X @ W.t())).sum()  # noqa: E731
    x64 = x.double()
    diff = (loss(x64 + v) - loss(x64 - v)) / 2
    size = (G.abs() @ W.abs() * v.abs()).sum()
    assert abs((dx.double() * v).sum() - diff) <= size * (2 * 128 + 16) * U
    X, G = value(xt8, k, m).t(), value(gt8, n, m).t()
    v = normal(5, (n, k)).double()
    loss = lambda W: (G * (X @ W.t())).sum()  # noqa: E731
    diff = (loss(w.double() + v) - loss(w.double() - v)) / 2
    size = (G.abs().t() @ X.abs() * v.abs()).sum()
    assert abs((dw.double() * v).sum() - diff) <= size * (2 * 128 + 16) * U


# ----------------------------------------------------------------- root-mean-square norm

COLS = [1, 8, 100, 128, 257, 768, 1001, 2048, 2056, 4096, 5000, 8192, 9001, 16384, 17000]


def chain(cols):
    """The longest fp32 sum of a row: a thread's run, the warp's and the CTA's tree."""
    return max(16, cols / 1024 + 8) + 5 + 32


@pytest.mark.parametrize("dtype,wdtype,f8", [(BF16, BF16, E4M3), (F16, F32, E5M2)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("cols", COLS)
def test_rmsnorm(cols, residual, dtype, wdtype, f8):
    rows = 5
    x, w = normal(1, (rows, cols), dtype), (1 + normal(2, (cols,), F32, 0.2)).to(wdtype)
    r = normal(3, (rows, cols), dtype, 2.0) if residual else None
    x[1] = 0.0
    if residual:
        r[1] = 0.0
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, s = zs.fp8_empty(rows, cols, f8)
    rstd = torch.empty(rows, device="cuda")
    zs.zero_rmsnorm_fp8(x, w, 1e-5, rstd, residual=r, h=h, y=y, q=q, s=s)
    want_h = (x.double() + (r.double() if residual else 0.0)).to(F32).to(dtype)
    assert torch.equal(h, want_h)
    rstd64, y64 = rmsnorm(h.double(), w.double(), 1e-5)
    rel = (chain(cols) / 2 + 4) * U
    assert ((rstd.double() - rstd64).abs() <= rstd64 * rel).all()
    assert ((y.double() - y64).abs() <= y64.abs() * (rel + 2 * U) + half_ulp(y64, dtype) * (1 + 1e-6)).all()
    check_blocks(y64, q, s, False, extra=2 * (rel + 2 * U), s_tol=rel + 3 * U)
    # each output alone: the same bits
    q2, s2 = zs.fp8_empty(rows, cols, f8)
    zs.zero_rmsnorm_fp8(x, w, 1e-5, residual=r, q=q2, s=s2)
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, s)
    # h over x itself
    y2 = torch.empty_like(y)
    zs.zero_rmsnorm_fp8(x, w, 1e-5, residual=r, h=x, y=y2)
    assert torch.equal(x, h) and torch.equal(y2, y)


@pytest.mark.parametrize("rows", [0, 1, 2, 700])
def test_rmsnorm_rows(rows):
    x, w = normal(1, (rows, 300), F16), normal(2, (300,), F16)
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    q, s = zs.fp8_empty(rows, 300)
    zs.zero_rmsnorm_fp8(x, w, 0.0, rstd, y=y, q=q, s=s)
    if rows:
        rstd64, y64 = rmsnorm(x.double(), w.double(), 0.0)
        rel = (chain(300) / 2 + 4) * U
        assert ((y.double() - y64).abs() <= y64.abs() * (rel + 2 * U) + half_ulp(y64, F16) * (1 + 1e-6)).all()
        check_blocks(y64, q, s, False, extra=2 * (rel + 2 * U), s_tol=rel + 3 * U)


@pytest.mark.parametrize("pad", [1, 8, 24])
def test_rmsnorm_strides_leave_the_gaps(pad):
    rows, cols = 9, 520
    nan = float("nan")
    x, r = (strided(normal(i, (rows, cols), BF16), pad, nan) for i in (1, 2))
    h, y = (strided(torch.zeros(rows, cols, dtype=BF16, device="cuda"), pad, 5.0) for _ in range(2))
    q = strided(torch.zeros(rows, cols, device="cuda").to(E4M3), pad, 5.0)
    s = strided(torch.zeros(5, rows, device="cuda"), pad, 5.0)
    w = normal(3, (cols,), BF16)
    rstd = torch.empty(rows, device="cuda")
    zs.zero_rmsnorm_fp8(x, w, 1e-6, rstd, residual=r, h=h, y=y, q=q, s=s)
    _, y64 = rmsnorm(h.double(), w.double(), 1e-6)
    rel = (chain(cols) / 2 + 4) * U
    assert ((y.double() - y64).abs() <= y64.abs() * (rel + 2 * U) + half_ulp(y64, BF16) * (1 + 1e-6)).all()
    check_blocks(y64, q, s, False, extra=2 * (rel + 2 * U), s_tol=rel + 3 * U)
    dy = strided(normal(4, (rows, cols), BF16), pad, nan)
    dx = strided(torch.zeros(rows, cols, dtype=BF16, device="cuda"), pad, 5.0)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, None, None)
    want, _, size, _ = rmsnorm_backward(dy.double(), h.double(), w.double(), rstd.double(), None)
    assert ((dx.double() - want).abs() <= size * chain(cols) * U + half_ulp(want, BF16) * (1 + 1e-6)).all()
    for t in (h, y, q, s, dx):
        assert (gap(t) == 5.0).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_rmsnorm_passes_on_what_is_not_finite(bad):
    x, w = normal(1, (4, 300), BF16), normal(2, (300,), BF16)
    x[2, 7] = bad
    y = torch.empty_like(x)
    q, s = zs.fp8_empty(4, 300)
    zs.zero_rmsnorm_fp8(x, w, 1e-5, y=y, q=q, s=s)
    v = q.double() * at_elements(s, 4, 300, False)
    ok = torch.tensor([0, 1, 3], device="cuda")
    assert y[ok].isfinite().all() and v[ok].isfinite().all()
    assert y[2, 7].isnan() and v[2, :128].isnan().all()


def backward_case(rows, cols, dtype, residual, seed=0):
    h, dy = normal(seed + 1, (rows, cols), dtype, 2.0), normal(seed + 2, (rows, cols), dtype)
    w = 1 + normal(seed + 3, (cols,), F32, 0.2)
    dr = normal(seed + 4, (rows, cols), dtype) if residual else None
    rstd = torch.rsqrt(h.double().square().mean(1) + 1e-5).float()
    return h, dy, w, dr, rstd


@pytest.mark.parametrize("dtype,dwt", [(BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("rows,cols", [(0, 40), (1, 1), (3, 100), (1000, 64), (37, 257), (700, 768), (9, 1001),
                                       (33, 2048), (20, 4096), (11, 5001), (6, 8192), (5, 9001)])
def test_rmsnorm_backward(rows, cols, residual, dtype, dwt):
    h, dy, w, dr, rstd = backward_case(rows, cols, dtype, residual)
    dx = torch.empty_like(h)
    dw = normal(9, (cols,), dwt)
    before = dw.double()
    ws = torch.empty(zs.zero_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda").fill_(255)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dr)
    want, want_w, size, size_w = rmsnorm_backward(dy.double(), h.double(), w.double(), rstd.double(),
                                                  dr.double() if residual else None)
    tol = size * (chain(cols) + 4) * U
    assert ((dx.double() - want).abs() <= tol + half_ulp(want, dtype) * (1 + 1e-6)).all()
    tol_w = size_w * (rows / 304 + 64) * U
    assert ((dw.double() - want_w).abs() <= tol_w + half_ulp(want_w, dwt) * (1 + 1e-6)).all()
    again = torch.empty_like(dw)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, again, ws, dres=dr)
    assert torch.equal(dw, again)
    dw.copy_(before)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dr, add_dw=True)
    sum_w = want_w + before
    assert ((dw.double() - sum_w).abs() <= tol_w + sum_w.abs() * U + half_ulp(sum_w, dwt) * (1 + 1e-6)).all()
    if rows:  # dx over dy itself
        over = dy.clone()
        zs.zero_rmsnorm_backward(over, h, w, rstd, over, None, None, dres=dr)
        assert torch.equal(over, dx)


def test_rmsnorm_backward_against_differences():
    """L = <dy, rmsnorm(h, w)> along random directions, central differences in
    64 bits (error of the order of the step squared)."""
    rows, cols = 6, 300
    h, dy, w, _, rstd = backward_case(rows, cols, BF16, False, seed=20)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(zs.zero_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws)
    h64, w64, dy64 = h.double(), w.double(), dy.double()
    vh, vw, e = normal(31, (rows, cols)).double(), normal(32, (cols,)).double(), 1e-5
    loss = lambda a, b: (dy64 * rmsnorm(a, b, 1e-5)[1]).sum()  # noqa: E731
    diff = (loss(h64 + e * vh, w64) - loss(h64 - e * vh, w64)) / (2 * e)
    room = (half_ulp(dx.double(), BF16) * 2 * vh.abs()).sum() + 1e-6 * (dx.double() * vh).abs().sum()
    assert abs((dx.double() * vh).sum() - diff) <= room
    diff = (loss(h64, w64 + e * vw) - loss(h64, w64 - e * vw)) / (2 * e)
    assert abs((dw.double() * vw).sum() - diff) <= 1e-5 * (dw.double() * vw).abs().sum()


# ----------------------------------------------------------------- streams, graphs, layouts

def test_operators_on_another_stream_and_in_a_graph():
    m, n, k = 40, 256, 384
    x, w = normal(1, (m, k), BF16), normal(2, (k,), BF16)
    wt = normal(3, (n, k), BF16, 0.1)
    y8, w8 = zs.fp8_empty(m, k), zs.fp8_empty(n, k, tile=True)
    rstd, out = torch.empty(m, device="cuda"), torch.empty(m, n, dtype=BF16, device="cuda")
    ws, stat = workspace(m, n, k), zs.new_tensors_stat()
    dx, dw = torch.empty_like(x), torch.empty(k, device="cuda")
    nws = torch.zeros(zs.zero_tensors_workspace_bytes([out, dw]), dtype=torch.uint8, device="cuda")
    rws = torch.empty(zs.zero_rmsnorm_workspace_bytes(m, k), dtype=torch.uint8, device="cuda")

    def go():
        zs.zero_fp8_quantize(wt, *w8, tile=True)
        zs.zero_rmsnorm_fp8(x, w, 1e-5, rstd, q=y8[0], s=y8[1])
        zs.zero_fp8_matmul(*y8, *w8, out, ws)
        zs.zero_rmsnorm_backward(x, x, w, rstd, dx, dw, rws)
        zs.zero_tensors_norm([out, dw], 1.0, stat, nws)
        zs.zero_tensors_clip([out], None, 1.0, 1.0, stat)

    go()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, dx, dw, stat)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        go()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, dx, dw, stat)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, dx, dw, stat)))


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """Rows more than 2^32 elements apart from the first one."""
    ld, rows, cols = (1 << 30) + 16, 5, 256
    big = torch.empty((rows - 1) * ld + cols, dtype=torch.uint8, device="cuda")
    a = torch.as_strided(big.view(E4M3), (rows, cols), (ld, 1))
    x = normal(1, (rows, cols), BF16)
    s = torch.empty(2, rows, device="cuda")
    zs.zero_fp8_quantize(x, a, s)
    check_blocks(x.double(), a, s, False)
    b, sb = operand(2, 130, cols, E4M3, True)
    out = torch.empty(rows, 130, device="cuda")
    zs.zero_fp8_matmul(a, s, b, sb, out, workspace(rows, 130, cols))
    check_product(out, a, s, b, sb)
    y = torch.as_strided(torch.empty((rows - 1) * ld + cols, dtype=BF16, device="cuda"), (rows, cols), (ld, 1))
    w = torch.ones(cols, device="cuda")
    zs.zero_rmsnorm_fp8(x, w, 0.0, y=y)
    _, y64 = rmsnorm(x.double(), w.double(), 0.0)
    assert ((y.double() - y64).abs() <= y64.abs() * 40 * U + half_ulp(y64, BF16) * (1 + 1e-6)).all()
