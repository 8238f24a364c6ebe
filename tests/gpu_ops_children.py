"""Child of test_gpu_ops_edges.py for the test setting that the operators'
library reads once per process (ZERO_TEST_MATMUL_GIVE_UP): prints one JSON line."""
import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

# k split over single CTAs, over clusters; single tokens and a tile to each CTA; CTAs that walk tiles; pairs
SIZES = [(512, 1024, 8192), (300, 700, 5000), (16, 4096, 14336), (40, 4096, 640), (1, 50257, 769), (128, 40000, 300),
         (1024, 4096, 1024)]


def give_up():
    """Every second CTA gives up: the error word is set, the counters are zero
    again, nothing outside the output is written and the process keeps using the GPU."""
    import torch
    import zero_partitioned_mixed_step_gb300 as zs
    assert os.environ["ZERO_TEST_MATMUL_GIVE_UP"] == "1"
    for m, n, k in SIZES:
        for tile in (True, False):
            (a, sa), (b, sb) = zs.fp8_empty(m, k), zs.fp8_empty(n, k, tile=tile)
            for t in (a, b):
                t.copy_(torch.ones(t.shape, device="cuda").to(t.dtype))
            sa.fill_(1.0)
            sb.fill_(1.0)
            out = torch.full((m, n + 16), 5.0, device="cuda", dtype=torch.bfloat16)
            ws = torch.zeros(zs.zero_fp8_matmul_workspace_bytes(m, n, k) + 64, dtype=torch.uint8, device="cuda")
            zs.zero_fp8_matmul(a, sa, b, sb, out[:, :n], ws[:-64])
            torch.cuda.synchronize()
            assert zs.read_matmul_error(ws) and int(ws[:4].view(torch.int32)) == 1, (m, n, k)
            assert int(ws[4:4096].sum()) == 0, (m, n, k, "counters")
            assert int(ws[-64:].sum()) == 0 and bool((out[:, n:] == 5).all()), (m, n, k)
    x = torch.arange(1 << 20, device="cuda", dtype=torch.int64)
    assert int(x.sum()) == (1 << 20) * ((1 << 20) - 1) // 2
    return {"ok": True}


if __name__ == "__main__":
    print(json.dumps({"give_up": give_up}[sys.argv[1]]()))
