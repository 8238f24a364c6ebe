"""Rows of several widths that one kernel serves, called from several threads and captured in one graph: how
much shared memory a launch takes is its own matter."""
import sys
import threading

import pytest
import torch

import zero_partitioned_mixed_step_gb300 as zs
from test_gpu_layer import BF16, E4M3, F32, backward_inputs, normal, run_backward, run_norms, same

pytestmark = pytest.mark.gpu

# each group of widths runs in one kernel, and takes a different amount of shared memory for each
GROUPS = [(2600, 4096, 2816, 3840), (1032, 2048, 1280, 1792), (2056, 2560, 2304, 2432), (4104, 8192, 5120, 6144)]


@pytest.mark.parametrize("widths", GROUPS)
@pytest.mark.parametrize("what", ["forward", "backward", "backward of halves"])
def test_widths_from_several_threads(widths, what):
    """Each thread's calls reach the library side by side: ctypes gives up the interpreter's lock."""
    rows, errors, barrier = 2, [], threading.Barrier(len(widths))
    w = torch.ones(max(widths), device="cuda")

    def work(cols):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                o = torch.ones(rows, cols, device="cuda", dtype=BF16)
                h, d_o, dx, r = torch.empty_like(o), torch.empty_like(o), torch.empty_like(o), torch.ones(rows, device="cuda")
                q, s = zs.fp8_empty(rows, cols)
                zs.zero_fp8_quantize(o, q, s)
                lib, check, raw = zs.layer.lib(), zs.layer.check, stream.cuda_stream
                m = (o.data_ptr(), cols)
                if what == "forward":
                    args = (*m, *m, None, w.data_ptr(), 4, None, 0, 4, 1.0, 1, rows, cols, 1e-5, h.data_ptr(), cols, None, 0,
                            8, None, None, None, None, None, raw)
                    call = lib.zero_gated_norms_fp8
                else:
                    kept = (*m, None, 0) if what.endswith("halves") else (q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0))
                    args = (*m, None, 0, *kept, *kept, None, r.data_ptr(), None, w.data_ptr(), 4, None, 0, 4, 1.0, 1, rows,
                            cols, d_o.data_ptr(), cols, dx.data_ptr(), cols, None, None, None, 4, 0, None, 0, raw)
                    call = lib.zero_gated_norms_backward
                stream.synchronize()
                barrier.wait(60)
                for i in range(15_000):
                    check(what, call(*args))
                stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append((cols, repr(e)))

    every = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(c,)) for c in widths]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(every)
    assert not errors


@pytest.mark.parametrize("s8", [True, False])
@pytest.mark.parametrize("widths", GROUPS)
def test_widths_in_one_graph(widths, s8):
    """Captured from the widest row to the narrowest and replayed: the bits of the calls one by one."""
    cases = [backward_inputs(5, c, BF16, F32, "cols", True, s8, seed=c) for c in sorted(widths, reverse=True)]
    x = [normal(c["dy"].shape[1], c["dy"].shape, BF16) for c in cases]

    def run():
        forward = [run_norms(c["dy"], t, c["w_pre"], c["w_post"], c["gate"], 1.0, E4M3) for c, t in zip(cases, x)]
        return forward, [run_backward(scale=1.0, **c) for c in cases]

    want = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip([*got[0], *got[1]], [*want[0], *want[1]]):
        for k in a:
            for p, q in zip(a[k], b[k]) if isinstance(a[k], tuple) else [(a[k], b[k])]:
                assert p is None or same(p, q), k
