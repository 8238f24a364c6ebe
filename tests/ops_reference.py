"""Plain 64-bit forms of the operators around the step, for the GPU tests."""
import math

import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
FRACTION = {torch.float8_e4m3fn: 3, torch.float8_e5m2: 2, torch.float16: 10, torch.bfloat16: 7,
            torch.float32: 23}
MIN_EXP = {torch.float8_e4m3fn: -6, torch.float8_e5m2: -14, torch.float16: -14,
           torch.bfloat16: -126, torch.float32: -126}
TINY = 2.0 ** -126
U = 2.0 ** -24  # half a unit in the last place of fp32


def half_ulp(x64, dtype):
    """Half the spacing of dtype's values at x64 (the largest error of rounding to nearest)."""
    e = torch.floor(torch.log2(x64.abs().clamp_min(2.0 ** MIN_EXP[dtype]))).clamp_min(MIN_EXP[dtype])
    return torch.exp2(e - FRACTION[dtype] - 1)


def blocks(n):
    return (n + 127) // 128


def block_amax(x64, tile):
    """[ceil(cols / 128), rows or ceil(rows / 128)] largest magnitudes."""
    r, k = x64.shape
    out = torch.zeros(blocks(k), blocks(r) if tile else r, dtype=torch.float64, device=x64.device)
    for j in range(blocks(k)):
        part = x64[:, 128 * j:128 * j + 128].abs()
        if tile:
            for i in range(blocks(r)):
                out[j, i] = part[128 * i:128 * i + 128].max()
        else:
            out[j] = part.max(1).values
    return out


def scales(x64, fp8, tile):
    return torch.clamp(block_amax(x64, tile) / QMAX[fp8], min=TINY)


def at_elements(s, rows, cols, tile):
    """Block scales at each element of [rows, cols]."""
    r = torch.arange(rows, device=s.device)
    c = torch.arange(cols, device=s.device)
    return s.double()[c[None, :] // 128, (r // 128 if tile else r)[:, None]]


def matmul(a, sa, b, sb):
    """The product in 64 bits, and the same sum over magnitudes."""
    n, k = b.shape
    a64 = a.double() * at_elements(sa, a.shape[0], k, False)
    b64 = b.double() * at_elements(sb, n, k, sb.shape[1] != n)
    return a64 @ b64.t(), a64.abs() @ b64.abs().t()


def rmsnorm(h64, w64, eps):
    rstd = 1.0 / torch.sqrt((h64 * h64).mean(1) + eps)
    return rstd, h64 * rstd[:, None] * w64


def rmsnorm_backward(dy64, h64, w64, rstd64, dres64):
    """dx, dw, and the sums of the magnitudes that each is made of."""
    xhat, g = h64 * rstd64[:, None], dy64 * w64
    m = (g * xhat).mean(1, keepdim=True)
    dx = rstd64[:, None] * (g - xhat * m)
    size = rstd64[:, None] * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if dres64 is not None:
        dx, size = dx + dres64, size + dres64.abs()
    return dx, (dy64 * xhat).sum(0), size, (dy64 * xhat).abs().sum(0)


def clip_factor(sumsq64, inv, max_norm):
    c = min(1.0, max_norm / (math.sqrt(sumsq64) + 1e-6)) if max_norm > 0 else 1.0
    return inv * c
