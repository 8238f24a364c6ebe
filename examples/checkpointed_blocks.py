"""Train feed-forward blocks whose backward pass reads 8-bit checkpoints, with the partitioned step.

Each block has a norm ahead of it and one behind, a learned gate for each channel and a
gated activation:
    y = norm(x) w_pre,  u | v = y up^T,  o = (silu(u) v) down^T,  x <- x + gate * norm(o) w_post
Between the products everything runs in the calls of zerostep_layer.h.  Of a block the
forward pass keeps o, x, u and v, each in 8 bits, and two numbers a token; the
backward pass makes the operands of its products from them:
  the norms' gradients from o and x,
  the activation's, in 8 bits along the row and along the tokens, from u and v,
  the transposed operand of up's gradient from x.

    python examples/checkpointed_blocks.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import zero_partitioned_mixed_step_gb300 as zs  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16 = torch.bfloat16


def half(*shape):
    return torch.empty(*shape, dtype=BF16, device="cuda")


class Blocks:
    """`depth` blocks on `tokens` rows and the norm behind the last; the buffers of one training step."""

    def __init__(self, tokens: int, d: int, ffn: int, depth: int, lr: float = 1e-3, max_norm: float = 1.0, seed: int = 0):
        if d % 16 or ffn % 128:
            raise ValueError("d: a multiple of 16, ffn: one of 128 (u and v share a matrix in blocks of 128) expected")
        self.tokens, self.d, self.ffn, self.depth, self.max_norm = tokens, d, ffn, depth, max_norm
        self.eps = 1e-5
        block = [(d,), (2 * ffn, d), (d, ffn), (d,), (d,)]  # w_pre, up, down, w_post, gate
        self.shapes = block * depth + [(d,)]
        self.step = zs.ZeroStep([torch.Size(s).numel() for s in self.shapes], 1, zs.BF16,
                                zs.adam_cfg(lr=lr, weight_decay=0.01))
        g = torch.Generator(device="cuda").manual_seed(seed)
        for i, w in enumerate(self.views(self.step.master[0])):
            if w.dim() == 1:
                w.fill_(0.5 if i % 5 == 4 and i < 5 * depth else 1.0)
            else:
                w.normal_(0.0, w.shape[1] ** -0.5, generator=g)
        self.step.params[0].copy_(self.step.master[0])
        self.params = [self.views(p) for p in self.step.params]  # of both slots
        self.flat_grad = torch.zeros(self.step.grad_numel(), dtype=BF16, device="cuda")
        self.grads = [half(*s) for s in self.shapes]
        self.grad_list = zs.tensor_list(self.grads)
        self.flat_list = zs.tensor_list([v.reshape(-1) for v in self.views(self.flat_grad)])
        self.stat = zs.new_tensors_stat()
        self.norm_ws = torch.zeros(zs.zero_tensors_workspace_bytes(self.grad_list), dtype=torch.uint8, device="cuda")
        sizes = [(tokens, 2 * ffn, d), (tokens, d, ffn), (tokens, ffn, d), (tokens, d, 2 * ffn), (2 * ffn, d, tokens),
                 (d, ffn, tokens)]
        self.mm_ws = torch.zeros(max(zs.zero_fp8_matmul_workspace_bytes(*s) for s in sizes), dtype=torch.uint8,
                                 device="cuda")
        self.gn_ws = torch.empty(zs.zero_gated_norms_workspace_bytes(tokens, d), dtype=torch.uint8, device="cuda")
        self.rms_ws = torch.empty(zs.zero_rmsnorm_workspace_bytes(tokens, d), dtype=torch.uint8, device="cuda")
        # what is kept of each block, and of the norm behind the last
        self.x8 = [zs.fp8_empty(tokens, d) for _ in range(depth + 1)]
        self.o8 = [zs.fp8_empty(tokens, d) for _ in range(depth)]
        self.u8 = [zs.fp8_empty(tokens, ffn) for _ in range(depth)]
        self.v8 = [zs.fp8_empty(tokens, ffn) for _ in range(depth)]
        self.rstd_pre = [torch.empty(tokens, device="cuda") for _ in range(depth + 1)]
        self.rstd_post = [torch.empty(tokens, device="cuda") for _ in range(depth)]
        # one block's
        self.x, self.y, self.o, self.uv = half(tokens, d), half(tokens, d), half(tokens, d), half(tokens, 2 * ffn)
        self.y8, self.a8 = zs.fp8_empty(tokens, d), zs.fp8_empty(tokens, ffn)
        self.up8, self.upt8 = zs.fp8_empty(2 * ffn, d, tile=True), zs.fp8_empty(d, 2 * ffn, tile=True)
        self.down8, self.downt8 = zs.fp8_empty(d, ffn, tile=True), zs.fp8_empty(ffn, d, tile=True)
        self.dy, self.d_o, self.dx, self.da = half(tokens, d), half(tokens, d), half(tokens, d), half(tokens, ffn)
        self.do8, self.do8t = zs.fp8_empty(tokens, d, E5M2), zs.fp8_empty(d, tokens, E5M2)
        self.duv8, self.duv8t = zs.fp8_empty(tokens, 2 * ffn, E5M2), zs.fp8_empty(2 * ffn, tokens, E5M2)
        self.a8t, self.y8t = zs.fp8_empty(ffn, tokens), zs.fp8_empty(d, tokens)

    def views(self, flat):
        return [flat[o:o + torch.Size(s).numel()].view(s) for o, s in zip(self.step.offsets, self.shapes)]

    def of_block(self, tensors, i):
        return tensors[5 * i:5 * i + 5]

    def forward(self, x, slot):
        """The normed stream behind the last block."""
        p, ffn = self.params[slot], self.ffn
        self.x0 = x
        zs.zero_rmsnorm_fp8(x, p[0], self.eps, self.rstd_pre[0], q=self.y8[0], s=self.y8[1])
        zs.zero_fp8_quantize(x, *self.x8[0])
        for i in range(self.depth):
            _, up, down, w_post, gate = self.of_block(p, i)
            zs.zero_fp8_quantize(up, *self.up8, tile=True)
            zs.zero_fp8_matmul(*self.y8, *self.up8, self.uv, self.mm_ws)
            zs.zero_activation_fp8(self.uv[:, :ffn], self.uv[:, ffn:], "silu", a8=self.a8, u8=self.u8[i], v8=self.v8[i])
            zs.zero_fp8_quantize(down, *self.down8, tile=True)
            zs.zero_fp8_matmul(*self.a8, *self.down8, self.o, self.mm_ws)
            last = i + 1 == self.depth
            zs.zero_gated_norms_fp8(self.o, x, p[5 * (i + 1)], self.eps, self.x, w_post=w_post, gate=gate,
                                    y=self.y if last else None, y8=None if last else self.y8, o8=self.o8[i],
                                    h8=self.x8[i + 1], rstd_post=self.rstd_post[i], rstd_pre=self.rstd_pre[i + 1])
            x = self.x
        return self.y

    def backward(self, dout, slot):
        """Gradients of the parameters and of the input for the gradient `dout` of forward()."""
        p, ffn, kb = self.params[slot], self.ffn, self.ffn // 128
        (duv, s_duv), (duvt, s_duvt) = self.duv8, self.duv8t
        dy, dx = dout, None
        for i in reversed(range(self.depth)):
            w_pre, up, down, w_post, gate = self.of_block(p, i)
            d_pre, d_up, d_down, d_post, d_gate = self.of_block(self.grads, i)
            zs.zero_gated_norms_backward(dy, self.o8[i][0], self.x8[i + 1][0], p[5 * (i + 1)], self.rstd_pre[i + 1],
                                         self.d_o, self.dx, self.gn_ws, so=self.o8[i][1], sh=self.x8[i + 1][1], dh=dx,
                                         w_post=w_post, rstd_post=self.rstd_post[i], gate=gate,
                                         dw_pre=self.grads[5 * (i + 1)], dw_post=d_post, dgate=d_gate)
            dx = self.dx
            zs.zero_fp8_quantize(down, None, None, *self.downt8, tile=True)
            zs.zero_fp8_quantize(self.d_o, *self.do8, *self.do8t)
            zs.zero_fp8_matmul(*self.do8, *self.downt8, self.da, self.mm_ws)
            zs.zero_activation_backward_fp8(self.da, self.u8[i][0], self.v8[i][0], "silu", su=self.u8[i][1],
                                            sv=self.v8[i][1], du8=(duv[:, :ffn], s_duv[:kb]),
                                            dv8=(duv[:, ffn:], s_duv[kb:]), du8t=(duvt[:ffn], s_duvt[:, :ffn]),
                                            dv8t=(duvt[ffn:], s_duvt[:, ffn:]), a8t=self.a8t)
            zs.zero_fp8_matmul(*self.do8t, *self.a8t, d_down, self.mm_ws)
            zs.zero_fp8_restore(*self.x8[i], row=self.rstd_pre[i], col=w_pre, t8=self.y8t)
            zs.zero_fp8_matmul(*self.duv8t, *self.y8t, d_up, self.mm_ws)
            zs.zero_fp8_quantize(up, None, None, *self.upt8, tile=True)
            zs.zero_fp8_matmul(*self.duv8, *self.upt8, self.dy, self.mm_ws)
            dy = self.dy
        zs.zero_rmsnorm_backward(dy, self.x0, p[0], self.rstd_pre[0], self.dx, self.grads[0], self.rms_ws, dres=dx)
        return self.dx

    def update(self):
        """The global norm, the clipped gradients into the flat buffer, the step."""
        zs.zero_tensors_norm(self.grad_list, 1.0, self.stat, self.norm_ws)
        zs.zero_tensors_clip(self.grad_list, self.flat_list, 1.0, self.max_norm, self.stat)
        self.step.step([self.flat_grad])


def train(blocks: Blocks, x, target, steps: int):
    """Mean squared error to `target`; (loss, gradient norm) of each step."""
    seen = []
    for _ in range(steps):
        slot = blocks.step.read_state().cur
        err = blocks.forward(x, slot).float() - target.float()
        loss = err.square().mean()
        blocks.backward((err * (2.0 / err.numel())).to(BF16), slot)
        blocks.update()
        if zs.read_matmul_error(blocks.mm_ws):
            raise RuntimeError("a product gave up waiting: its output is undefined")
        seen.append((float(loss), zs.read_tensors_stat(blocks.stat).norm))
    return seen


def main(steps: int = 20):
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens, d, ffn, depth = 2048, 1024, 2048, 4
    x, target = (torch.randn(tokens, d, device="cuda", generator=g).to(BF16) for _ in range(2))
    for i, (loss, norm) in enumerate(train(Blocks(tokens, d, ffn, depth), x, target, steps)):
        print(f"step {i + 1:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main(*map(int, sys.argv[1:]))
