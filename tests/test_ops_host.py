"""libzerostep_ops.so on the host, without a GPU: it exports what
include/zerostep_ops.h declares and nothing else, and its entry points refuse
invalid arguments before anything is enqueued (this machine has no device, so
a launch would fail with a CUDA error instead)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "zerostep_ops.h")
EINVAL, EALIGN, ESPACE = -1, -2, -3
F16, BF16, F32, E4M3, E5M2 = 0, 1, 4, 8, 9
P = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from zero_partitioned_mixed_step_gb300 import _build, _ops_abi
    _build.build()
    return _ops_abi.lib()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return set(re.findall(r"\b(zero_\w+)\s*\(", text))


def test_exports_what_the_header_declares(lib):
    from zero_partitioned_mixed_step_gb300 import _build, _ops_abi
    assert declared() == set(_ops_abi.SIGNATURES) and len(declared()) == 9
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("nm not installed")
    out = subprocess.run([nm, "-D", "--defined-only", _build.OPS_LIB], capture_output=True,
                         text=True, check=True).stdout
    assert {ln.split()[-1] for ln in out.splitlines() if ln.strip()} - {"_init", "_fini"} == declared()


def test_stat_matches_the_header(tmp_path, lib):
    from zero_partitioned_mixed_step_gb300 import _ops_abi
    src = tmp_path / "off.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "zerostep_ops.h"\nint main(void)'
                   '{printf("%zu %zu %zu %zu %d %d %d %d %d", sizeof(zero_tensors_stat),'
                   "offsetof(zero_tensors_stat, sumsq), offsetof(zero_tensors_stat, norm),"
                   "offsetof(zero_tensors_stat, found_inf), ZERO_T_F16, ZERO_T_BF16, ZERO_T_F32,"
                   "ZERO_T_E4M3, ZERO_T_E5M2);return 0;}")
    exe = tmp_path / "off"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    S = _ops_abi.TensorsStat
    assert got == [ctypes.sizeof(S), S.sumsq.offset, S.norm.offset, S.found_inf.offset,
                   F16, BF16, F32, E4M3, E5M2]


def _list(ptrs, numels, types):
    n = len(ptrs)
    return ((ctypes.c_void_p * max(n, 1))(*ptrs), (ctypes.c_int64 * max(n, 1))(*numels),
            (ctypes.c_int32 * max(n, 1))(*types))


def test_tensors_norm_refuses(lib):
    def call(ptrs=(P,), numels=(10,), types=(BF16,), inv=1.0, sumsq=None, stat=P, ws=P, ws_bytes=1 << 20):
        x, k, t = _list(ptrs, numels, types)
        return lib.zero_tensors_norm(len(ptrs), x, k, t, inv, sumsq, stat, ws, ws_bytes, None)

    assert call(numels=(-1,)) == EINVAL and call(types=(E4M3,)) == EINVAL
    assert call(ptrs=(None,)) == EINVAL and call(stat=None) == EINVAL and call(ws=None) == EINVAL
    for inv in (0.0, -1.0, float("inf"), float("nan")):
        assert call(inv=inv) == EINVAL
    assert call(ptrs=(P + 1,)) == EALIGN and call(ptrs=(P + 2,), types=(F32,)) == EALIGN
    assert call(stat=P + 4) == EALIGN and call(sumsq=P + 4) == EALIGN and call(ws=P + 8) == EALIGN
    assert call(ws_bytes=8) == ESPACE
    assert lib.zero_tensors_norm(-1, None, None, None, 1.0, None, P, P, 1 << 20, None) == EINVAL
    assert lib.zero_tensors_norm(1, None, None, None, 1.0, None, P, P, 1 << 20, None) == EINVAL


def test_tensors_workspace(lib):
    def need(*numels):
        return lib.zero_tensors_workspace_bytes(len(numels), _list([0] * len(numels), numels, [0])[1])

    assert need() == 256 and need(0, 0) == 256 and need(1) == 264
    assert need(4096) == 264 and need(4097) == 272 and need(4096, 1) == 272
    assert need(8_030_261_248) <= 256 + 8 * 16385
    assert need(-1) == 0 and lib.zero_tensors_workspace_bytes(-1, None) == 0


def test_tensors_clip_refuses(lib):
    def call(ptrs=(P,), numels=(10,), types=(BF16,), outs=None, otypes=None, inv=1.0, most=1.0, stat=P):
        x, k, t = _list(ptrs, numels, types)
        o = _list(outs, numels, otypes or types) if outs is not None else (None, None, None)
        return lib.zero_tensors_clip(len(ptrs), x, k, t, o[0], o[2] if otypes is not False else None,
                                     inv, most, stat, None)

    assert call(most=-1.0) == EINVAL and call(most=float("nan")) == EINVAL and call(inv=0.0) == EINVAL
    assert call(stat=None) == EINVAL and call(stat=P + 4) == EALIGN
    assert call(outs=(None,)) == EINVAL and call(outs=(P + 1,)) == EALIGN
    assert call(outs=(P,), otypes=(F32,)) == EINVAL       # in place, another type
    assert call(outs=(P + 64,), otypes=(E5M2,)) == EINVAL and call(outs=(P + 64,), otypes=False) == EINVAL
    assert call(numels=(0,)) == 0                          # nothing to do


def test_quantize_refuses(lib):
    def call(x=P, t=BF16, rows=4, cols=130, ldx=130, f8=E4M3, tile=0, q=P, ldq=130, s=P, lds=4, qt=None,
             ldqt=4, st=None, ldst=130):
        return lib.zero_fp8_quantize(x, t, rows, cols, ldx, f8, tile, q, ldq, s, lds, qt, ldqt, st,
                                     ldst, None)

    assert call(t=E4M3) == EINVAL and call(f8=BF16) == EINVAL and call(rows=-1) == EINVAL
    assert call(cols=1 << 31) == EINVAL and call(tile=2) == EINVAL and call(x=None) == EINVAL
    assert call(ldx=129) == EINVAL and call(ldq=129) == EINVAL and call(lds=3) == EINVAL
    assert call(q=None) == EINVAL and call(s=None) == EINVAL and call(q=None, s=None) == EINVAL
    assert call(qt=P) == EINVAL and call(qt=P, st=P, ldqt=3) == EINVAL
    assert call(qt=P, st=P, ldst=129) == EINVAL
    assert call(x=P + 1) == EALIGN and call(s=P + 2) == EALIGN and call(t=F32, x=P + 2) == EALIGN
    assert call(rows=0) == 0 and call(cols=0) == 0


def test_matmul_refuses(lib):
    need = lib.zero_fp8_matmul_workspace_bytes(8, 130, 256)
    assert need > 0 and lib.zero_fp8_matmul_workspace_bytes(-1, 1, 1) == 0

    def call(a=P, at=E4M3, lda=256, sa=P, ldsa=8, b=P, bt=E5M2, ldb=256, sb=P, ldsb=2, tile=1, out=P,
             ot=BF16, ldo=130, m=8, n=130, k=256, ws=P, ws_bytes=need):
        return lib.zero_fp8_matmul(a, at, lda, sa, ldsa, b, bt, ldb, sb, ldsb, tile, out, ot, ldo, m,
                                   n, k, 0, ws, ws_bytes, None)

    assert call(at=BF16) == EINVAL and call(bt=F32) == EINVAL and call(ot=E4M3) == EINVAL
    assert call(m=-1) == EINVAL and call(n=(1 << 31) - 1) == EINVAL and call(k=-1) == EINVAL
    assert call(tile=2) == EINVAL and call(ws=None) == EINVAL and call(a=None) == EINVAL
    assert call(lda=255) == EINVAL and call(ldb=240) == EINVAL and call(ldo=129) == EINVAL
    assert call(ldsa=7) == EINVAL and call(ldsb=1) == EINVAL and call(tile=0) == EINVAL
    assert call(a=P + 8) == EALIGN and call(lda=264) == EALIGN and call(ldb=257) == EALIGN
    assert call(out=P + 1) == EALIGN and call(sa=P + 2) == EALIGN and call(ws=P + 8) == EALIGN
    assert call(ws_bytes=need - 1) == ESPACE
    assert call(m=0) == 0 and call(n=0) == 0


def test_rmsnorm_refuses(lib):
    def fwd(x=P, ldx=65, r=None, ldr=65, w=P, wt=F32, t=BF16, rows=3, cols=65, eps=1e-5, h=None, ldh=65,
            y=None, ldy=65, f8=E4M3, q=P, ldq=65, s=P, lds=3, rstd=None):
        return lib.zero_rmsnorm_fp8(x, ldx, r, ldr, w, wt, t, rows, cols, eps, h, ldh, y, ldy, f8, q,
                                    ldq, s, lds, rstd, None)

    assert fwd(t=F32) == EINVAL and fwd(wt=E4M3) == EINVAL and fwd(cols=0) == EINVAL
    assert fwd(eps=-1.0) == EINVAL and fwd(eps=float("nan")) == EINVAL and fwd(w=None) == EINVAL
    assert fwd(s=None) == EINVAL and fwd(f8=BF16) == EINVAL and fwd(q=None, s=None) == EINVAL
    assert fwd(ldx=64) == EINVAL and fwd(x=None) == EINVAL and fwd(lds=2) == EINVAL
    assert fwd(r=P, ldr=64) == EINVAL and fwd(h=P, ldh=1) == EINVAL and fwd(y=P, ldy=1) == EINVAL
    assert fwd(x=P + 1) == EALIGN and fwd(w=P + 2) == EALIGN and fwd(rstd=P + 2) == EALIGN
    assert fwd(rows=0) == 0

    need = lib.zero_rmsnorm_workspace_bytes(3, 65)
    assert need == 3 * 65 * 4 and lib.zero_rmsnorm_workspace_bytes(3, 0) == 0

    def bwd(dy=P, lddy=65, h=P, ldh=65, w=P, wt=F32, rstd=P, dr=None, lddr=65, t=F16, rows=3, cols=65,
            dx=P, lddx=65, dw=P, dwt=F32, ws=P, ws_bytes=need):
        return lib.zero_rmsnorm_backward(dy, lddy, h, ldh, w, wt, rstd, dr, lddr, t, rows, cols, dx,
                                         lddx, dw, dwt, 0, ws, ws_bytes, None)

    assert bwd(t=F32) == EINVAL and bwd(dwt=E4M3) == EINVAL and bwd(wt=E5M2) == EINVAL
    assert bwd(rstd=None) == EINVAL and bwd(w=None) == EINVAL and bwd(ws=None) == EINVAL
    assert bwd(dy=None) == EINVAL and bwd(h=None) == EINVAL and bwd(dx=None) == EINVAL
    assert bwd(lddy=64) == EINVAL and bwd(ldh=64) == EINVAL and bwd(lddx=64) == EINVAL
    assert bwd(dr=P, lddr=64) == EINVAL and bwd(rows=-1) == EINVAL
    assert bwd(dy=P + 1) == EALIGN and bwd(dw=P + 2) == EALIGN and bwd(ws=P + 8) == EALIGN
    assert bwd(ws_bytes=need - 1) == ESPACE


def test_binding_refuses_cpu_tensors(lib):
    import torch
    import zero_partitioned_mixed_step_gb300 as zs
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        zs.tensor_list([x])
    with pytest.raises(ValueError):
        zs.zero_fp8_quantize(x, None, None)
    with pytest.raises(ValueError):
        zs.zero_rmsnorm_fp8(x, torch.zeros(127), 1e-5)
    with pytest.raises(TypeError):
        zs.zero_fp8_matmul(x, x, x, x, x, x)
