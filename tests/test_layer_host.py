"""libzerostep_layer.so on the host, without a GPU: it exports what
include/zerostep_layer.h declares and nothing else, and its entry points refuse
invalid arguments before anything is enqueued."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "zerostep_layer.h")
EINVAL, EALIGN, ESPACE = -1, -2, -3
F16, BF16, F32, E4M3, E5M2 = 0, 1, 4, 8, 9
NONE, ONE, COLS, ROWS = 0, 1, 2, 3
P = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from zero_partitioned_mixed_step_gb300 import _build, _layer_abi
    _build.build()
    return _layer_abi.lib()


def form(q=P, ld=130, s=P, lds=4):
    from zero_partitioned_mixed_step_gb300._layer_abi import Fp8Form
    return ctypes.byref(Fp8Form(q, ld, s, lds))


def test_exports_what_the_header_declares(lib):
    from zero_partitioned_mixed_step_gb300 import _build, _layer_abi
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(zero_\w+)\s*\(", text))
    assert declared == set(_layer_abi.SIGNATURES)
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("nm not installed")
    out = subprocess.run([nm, "-D", "--defined-only", _build.LAYER_LIB], capture_output=True, text=True,
                         check=True).stdout
    assert {ln.split()[-1] for ln in out.splitlines() if ln.strip()} - {"_init", "_fini"} == declared


def test_header_is_c_and_matches_the_binding(tmp_path, lib):
    from zero_partitioned_mixed_step_gb300 import _layer_abi as abi
    src = tmp_path / "off.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "zerostep_layer.h"\nint main(void)'
                   '{printf("%zu %zu %zu %zu %zu %d %d %d %d %d %d", sizeof(zero_fp8_form), offsetof(zero_fp8_form, q),'
                   "offsetof(zero_fp8_form, ld), offsetof(zero_fp8_form, s), offsetof(zero_fp8_form, lds),"
                   "ZERO_GATE_NONE, ZERO_GATE_ONE, ZERO_GATE_COLS, ZERO_GATE_ROWS, ZERO_ACT_SILU, ZERO_ACT_GELU);"
                   "return 0;}")
    exe = tmp_path / "off"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    f = abi.Fp8Form
    assert got == [ctypes.sizeof(f), f.q.offset, f.ld.offset, f.s.offset, f.lds.offset, abi.GATE_NONE, abi.GATE_ONE,
                   abi.GATE_COLS, abi.GATE_ROWS, abi.ACT_SILU, abi.ACT_GELU]


def test_norms_refuse(lib):
    def call(o=P, ldo=130, x=P, ldx=130, wo=P, wp=P, wt=F32, g=P, gk=COLS, gt=F32, scale=1.0, t=BF16, rows=4, cols=130,
             eps=1e-5, h=P, ldh=130, y=None, ldy=130, f8=E4M3, y8=form(), o8=form(), h8=form(), ro=P, rp=P):
        return lib.zero_gated_norms_fp8(o, ldo, x, ldx, wo, wp, wt, g, gk, gt, scale, t, rows, cols, eps, h, ldh, y, ldy,
                                        f8, y8, o8, h8, ro, rp, None)

    assert call(t=F32) == EINVAL and call(wt=E4M3) == EINVAL and call(cols=0) == EINVAL and call(rows=-1) == EINVAL
    assert call(cols=1 << 31) == EINVAL and call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL
    assert call(scale=float("inf")) == EINVAL and call(scale=float("nan")) == EINVAL
    assert call(gk=4) == EINVAL and call(gk=-1) == EINVAL and call(g=None) == EINVAL and call(gt=E4M3) == EINVAL
    assert call(f8=BF16) == EINVAL and call(wp=None) == EINVAL
    assert call(o=None) == EINVAL and call(x=None) == EINVAL and call(h=None) == EINVAL
    assert call(ldo=129) == EINVAL and call(ldx=129) == EINVAL and call(ldh=129) == EINVAL
    assert call(y=P, ldy=129) == EINVAL
    for bad in (form(q=None), form(s=None), form(ld=129), form(lds=3)):
        assert call(y8=bad) == EINVAL and call(o8=bad) == EINVAL and call(h8=bad) == EINVAL
    assert call(o=P + 1) == EALIGN and call(wp=P + 2) == EALIGN and call(wo=P + 2) == EALIGN and call(g=P + 2) == EALIGN
    assert call(ro=P + 2) == EALIGN and call(rp=P + 2) == EALIGN and call(y8=form(s=P + 2)) == EALIGN
    assert call(rows=0) == 0


def test_norms_backward_refuses(lib):
    need = lib.zero_gated_norms_workspace_bytes(4, 130)
    assert need == (2 * 130 + 1) * 4
    assert lib.zero_gated_norms_workspace_bytes(-1, 8) == 0 and lib.zero_gated_norms_workspace_bytes(4, 0) == 0

    def call(dy=P, lddy=130, dh=P, lddh=130, o=P, ldo=130, so=P, ldso=4, h=P, ldh=130, sh=P, ldsh=4, ro=P, rp=P, wo=P,
             wp=P, wt=F32, g=P, gk=COLS, gt=F32, scale=1.0, t=BF16, rows=4, cols=130, d_o=P, lddo=130, dx=P, lddx=130,
             dwo=P, dwp=P, dg=P, dt=F32, ws=P, ws_bytes=need):
        return lib.zero_gated_norms_backward(dy, lddy, dh, lddh, o, ldo, so, ldso, h, ldh, sh, ldsh, ro, rp, wo, wp, wt,
                                             g, gk, gt, scale, t, rows, cols, d_o, lddo, dx, lddx, dwo, dwp, dg, dt, 0,
                                             ws, ws_bytes, None)

    assert call(t=F32) == EINVAL and call(wt=E5M2) == EINVAL and call(dt=E4M3) == EINVAL and call(cols=0) == EINVAL
    assert call(so=None) == EINVAL and call(sh=None) == EINVAL and call(ro=None) == EINVAL and call(rp=None) == EINVAL
    assert call(wo=None) == EINVAL                      # dw_post without w_post
    assert call(g=None, gk=NONE) == EINVAL              # dgate without a gate
    assert call(g=None) == EINVAL and call(gk=9) == EINVAL and call(wp=None) == EINVAL and call(ws=None) == EINVAL
    assert call(dy=None) == EINVAL and call(o=None) == EINVAL and call(h=None) == EINVAL
    assert call(d_o=None) == EINVAL and call(dx=None) == EINVAL and call(scale=float("nan")) == EINVAL
    for ld in ("lddy", "lddh", "ldo", "ldh", "lddo", "lddx"):
        assert call(**{ld: 129}) == EINVAL
    assert call(ldso=3) == EINVAL and call(ldsh=3) == EINVAL
    assert call(so=None, sh=None, o=P + 1) == EALIGN
    assert call(dy=P + 1) == EALIGN and call(so=P + 2) == EALIGN and call(dwp=P + 2) == EALIGN and call(dg=P + 1) == EALIGN
    assert call(ws=P + 16) == EALIGN and call(ws_bytes=need - 1) == ESPACE


def test_activation_refuses(lib):
    def fwd(u=P, ldu=130, v=P, ldv=130, act=0, t=BF16, rows=4, cols=130, a=P, lda=130, f8=E4M3, a8=form(), u8=form(),
            v8=form()):
        return lib.zero_activation_fp8(u, ldu, v, ldv, act, t, rows, cols, a, lda, f8, a8, u8, v8, None)

    assert fwd(t=F32) == EINVAL and fwd(act=2) == EINVAL and fwd(act=-1) == EINVAL and fwd(f8=BF16) == EINVAL
    assert fwd(v=None) == EINVAL                        # a checkpoint of what is not there
    assert fwd(u=None) == EINVAL and fwd(ldu=129) == EINVAL and fwd(ldv=129) == EINVAL and fwd(lda=129) == EINVAL
    assert fwd(a=None, a8=None, u8=None, v8=None) == EINVAL
    for bad in (form(q=None), form(s=None), form(ld=129), form(lds=3)):
        assert fwd(a8=bad) == EINVAL and fwd(u8=bad) == EINVAL and fwd(v8=bad) == EINVAL
    assert fwd(u=P + 1) == EALIGN and fwd(a=P + 1) == EALIGN and fwd(a8=form(s=P + 2)) == EALIGN
    assert fwd(rows=0) == 0 and fwd(cols=0) == 0 and fwd(rows=-1) == EINVAL

    t_form = form(ld=4, lds=130)

    def bwd(da=P, ldda=130, u=P, ldu=130, su=P, ldsu=4, v=P, ldv=130, sv=P, ldsv=4, act=1, t=F16, rows=4, cols=130,
            du=P, lddu=130, dv=P, lddv=130, f8=E5M2, du8=form(), dv8=form(), du8t=t_form, dv8t=t_form, a8t=t_form):
        return lib.zero_activation_backward_fp8(da, ldda, u, ldu, su, ldsu, v, ldv, sv, ldsv, act, t, rows, cols, du,
                                                lddu, dv, lddv, f8, du8, dv8, du8t, dv8t, a8t, None)

    assert bwd(t=F32) == EINVAL and bwd(act=7) == EINVAL and bwd(f8=F16) == EINVAL
    assert bwd(su=None) == EINVAL and bwd(sv=None) == EINVAL and bwd(v=None) == EINVAL
    assert bwd(v=None, sv=None) == EINVAL               # dv without v
    assert bwd(du=None, dv=None, du8=None, dv8=None, du8t=None, dv8t=None, a8t=None) == EINVAL
    for ld in ("ldda", "ldu", "ldv", "lddu", "lddv"):
        assert bwd(**{ld: 129}) == EINVAL
    assert bwd(ldsu=3) == EINVAL and bwd(ldsv=3) == EINVAL
    for bad in (form(q=None, ld=4, lds=130), form(ld=3, lds=130), form(ld=4, lds=129)):
        assert bwd(du8t=bad) == EINVAL and bwd(dv8t=bad) == EINVAL and bwd(a8t=bad) == EINVAL
    assert bwd(da=P + 1) == EALIGN and bwd(su=P + 1) == EALIGN and bwd(su=None, sv=None, u=P + 1) == EALIGN
    assert bwd(rows=0) == 0 and bwd(cols=0) == 0


def test_restore_refuses(lib):
    t_form = form(ld=4, lds=130)

    def call(q=P, f8=E4M3, ldq=130, s=P, lds=4, row=P, col=P, ct=F32, rows=4, cols=130, x=P, xt=BF16, ldx=130, t8=t_form):
        return lib.zero_fp8_restore(q, f8, ldq, s, lds, row, col, ct, rows, cols, x, xt, ldx, t8, None)

    assert call(f8=BF16) == EINVAL and call(ct=E4M3) == EINVAL and call(xt=E4M3) == EINVAL and call(rows=-1) == EINVAL
    assert call(q=None) == EINVAL and call(s=None) == EINVAL and call(x=None, t8=None) == EINVAL
    assert call(ldq=129) == EINVAL and call(lds=3) == EINVAL and call(ldx=129) == EINVAL
    assert call(t8=form(ld=3, lds=130)) == EINVAL and call(t8=form(ld=4, lds=129)) == EINVAL
    assert call(row=P + 2) == EALIGN and call(col=P + 2) == EALIGN and call(x=P + 1) == EALIGN and call(s=P + 1) == EALIGN
    assert call(rows=0) == 0 and call(cols=0) == 0


def test_binding_refuses(lib):
    import torch
    import zero_partitioned_mixed_step_gb300 as zs
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w, r = torch.ones(128), torch.ones(4)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(1, 4)
    with pytest.raises(ValueError):  # not on a GPU
        zs.zero_gated_norms_fp8(x, x, w, 1e-5, x)
    with pytest.raises(ValueError):
        zs.zero_activation_fp8(x, x, "silu", a=x)
    with pytest.raises(ValueError):
        zs.zero_fp8_restore(q, s, x=x)
    with pytest.raises(ValueError):
        zs.zero_gated_norms_backward(x, x, x, w, r, x, x, None, so=s)
    with pytest.raises(ValueError):
        zs.zero_gated_norms_backward(x, x, x, w, r, x, x, None, w_post=w)
    with pytest.raises(ValueError):
        zs.zero_gated_norms_backward(x, x, x, w, r, x, x, None, dgate=w)
    with pytest.raises(ValueError):
        zs.zero_activation_fp8(x, None, "silu", v8=(q, s))
    with pytest.raises(ValueError):
        zs.zero_activation_backward_fp8(x, x, None, "silu", dv=x)
    with pytest.raises(ValueError):
        zs.layer._act("relu")
    with pytest.raises(ValueError):
        zs.layer._gate_kind(torch.ones(5), 4, 128)
    with pytest.raises(TypeError):
        zs.layer._one_type((q, s), (x.to(torch.float8_e5m2), s))
    assert zs.layer._gate_kind(None, 4, 128) == NONE and zs.layer._gate_kind(torch.ones(1), 4, 128) == ONE
    assert zs.layer._gate_kind(w, 4, 128) == COLS and zs.layer._gate_kind(torch.ones(4, 1), 4, 128) == ROWS
