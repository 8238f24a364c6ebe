"""Entry points of libzerostep_ops.so at the edges of their arguments, without a GPU."""
import ctypes
import itertools

import pytest

E4M3, F32 = 8, 4
P = 1 << 20  # never dereferenced: there is nothing to compute


@pytest.fixture(scope="module")
def lib():
    from zero_partitioned_mixed_step_gb300 import _build, _ops_abi
    _build.build()
    return _ops_abi.lib()


def test_matmul_workspace_of_empty_sizes(lib):
    """Any of the sizes may be 0: the header of the workspace is what is needed."""
    for m, n, k in itertools.product((0, 1, 5, 64, 65, 300, 40000), (0, 1, 129, 50257), (0, 1, 769)):
        need = lib.zero_fp8_matmul_workspace_bytes(m, n, k)
        assert need >= 4096
        if m == 0 or n == 0:
            assert need == 4096
            assert lib.zero_fp8_matmul(P, E4M3, 784, P, max(m, 1), P, E4M3, 784, P, max(n, 1), 0, P, F32, max(n, 1),
                                       m, n, k, 0, P, need, None) == 0


def test_matmul_error_is_read():
    import torch
    import zero_partitioned_mixed_step_gb300 as zs
    ws = torch.zeros(4096, dtype=torch.uint8)
    ws[256:] = 1  # what follows the word is not read
    assert zs.read_matmul_error(ws) is False
    ws[:4].view(torch.int32).fill_(1)
    assert zs.read_matmul_error(ws) is True
    assert zs.read_matmul_error(ws.view(torch.float32)) is True
    ws[:4].zero_()
    assert zs.read_matmul_error(ws) is False
    with pytest.raises(ValueError):
        zs.read_matmul_error(ws[:2])
    with pytest.raises(ValueError):
        zs.read_matmul_error(ws[::2])
