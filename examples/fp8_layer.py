"""Train one feed-forward layer with 8-bit products and the partitioned step.

The parameters live in the step's flat bf16 buffer.  Each iteration
  casts the two weights to 8 bits in 128x128 tiles, with their transposes,
  runs  h = x + residual,  y = rmsnorm(h)  ->  up  ->  silu  ->  down,
  makes the gradients: the inputs' from the transposed weights, the weights'
  along the tokens, the norm's,
  takes the global norm over the three gradients and writes them, clipped,
  into the flat gradient buffer, and
  runs the step (AdamW on the fp32 master weights, cast back to bf16).

    python examples/fp8_layer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import zero_partitioned_mixed_step_gb300 as zs  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


class Layer:
    """rmsnorm -> up (ffn, d) -> silu -> down (d, ffn) on `tokens` rows, the
    buffers of one training step."""

    def __init__(self, tokens: int, d: int, ffn: int, lr: float = 1e-3, max_norm: float = 1.0, seed: int = 0):
        self.tokens, self.d, self.ffn, self.max_norm = tokens, d, ffn, max_norm
        self.eps = 1e-5
        shapes = [(d,), (ffn, d), (d, ffn)]
        numels = [torch.Size(s).numel() for s in shapes]
        self.step = zs.ZeroStep(numels, 1, zs.BF16, zs.adam_cfg(lr=lr, weight_decay=0.01))
        g = torch.Generator(device="cuda").manual_seed(seed)
        views = self.views(self.step.master[0], shapes)
        views[0].fill_(1.0)
        for w in views[1:]:
            w.normal_(0.0, w.shape[1] ** -0.5, generator=g)
        self.step.params[0].copy_(self.step.master[0])
        self.params = [self.views(p, shapes) for p in self.step.params]  # of both slots
        self.flat_grad = torch.zeros(self.step.grad_numel(), dtype=torch.bfloat16, device="cuda")
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.grads = [torch.empty(s, **bf16) for s in shapes]
        self.grad_list = zs.tensor_list(self.grads)
        self.flat_list = zs.tensor_list([v.reshape(-1) for v in self.views(self.flat_grad, shapes)])
        self.stat = zs.new_tensors_stat()
        self.norm_ws = torch.zeros(zs.zero_tensors_workspace_bytes(self.grad_list), dtype=torch.uint8, device="cuda")
        self.rms_ws = torch.empty(zs.zero_rmsnorm_workspace_bytes(tokens, d), dtype=torch.uint8, device="cuda")
        sizes = [(tokens, ffn, d), (tokens, d, ffn), (ffn, d, tokens), (d, ffn, tokens)]
        self.mm_ws = torch.zeros(max(zs.zero_fp8_matmul_workspace_bytes(*s) for s in sizes), dtype=torch.uint8,
                                 device="cuda")
        # activations: what the forward pass keeps, and their 8-bit forms
        self.h, self.y, self.out = (torch.empty(tokens, d, **bf16) for _ in range(3))
        self.u = torch.empty(tokens, ffn, **bf16)
        self.rstd = torch.empty(tokens, device="cuda")
        self.y8, self.a8 = zs.fp8_empty(tokens, d), zs.fp8_empty(tokens, ffn)
        self.yt8, self.at8 = zs.fp8_empty(d, tokens), zs.fp8_empty(ffn, tokens)
        self.up8, self.upt8 = zs.fp8_empty(ffn, d, tile=True), zs.fp8_empty(d, ffn, tile=True)
        self.down8, self.downt8 = zs.fp8_empty(d, ffn, tile=True), zs.fp8_empty(ffn, d, tile=True)
        # gradients in the wider range of E5M2
        self.do8, self.dot8 = zs.fp8_empty(tokens, d, E5M2), zs.fp8_empty(d, tokens, E5M2)
        self.du8, self.dut8 = zs.fp8_empty(tokens, ffn, E5M2), zs.fp8_empty(ffn, tokens, E5M2)
        self.da, self.dy = torch.empty(tokens, ffn, **bf16), torch.empty(tokens, d, **bf16)
        self.dx = torch.empty(tokens, d, **bf16)

    def views(self, flat, shapes):
        return [flat[o:o + torch.Size(s).numel()].view(s) for o, s in zip(self.step.offsets, shapes)]

    def forward(self, x, residual, slot):
        w_norm, up, down = self.params[slot]
        zs.zero_fp8_quantize(up, *self.up8, *self.upt8, tile=True)
        zs.zero_fp8_quantize(down, *self.down8, *self.downt8, tile=True)
        zs.zero_rmsnorm_fp8(x, w_norm, self.eps, self.rstd, residual=residual, h=self.h, y=self.y, q=self.y8[0],
                            s=self.y8[1])
        zs.zero_fp8_matmul(*self.y8, *self.up8, self.u, self.mm_ws)
        self.a = torch.nn.functional.silu(self.u)
        zs.zero_fp8_quantize(self.a, *self.a8, *self.at8)
        zs.zero_fp8_matmul(*self.a8, *self.down8, self.out, self.mm_ws)
        return self.out + self.h

    def backward(self, dout, slot):
        """Gradients of the three parameters and of x for the gradient `dout` of forward()."""
        dw_norm, dup, ddown = self.grads
        zs.zero_fp8_quantize(dout, *self.do8, *self.dot8)
        zs.zero_fp8_matmul(*self.do8, *self.downt8, self.da, self.mm_ws)
        zs.zero_fp8_matmul(*self.dot8, *self.at8, ddown, self.mm_ws)
        s = torch.sigmoid(self.u.float())
        du = (self.da * (s * (1 + self.u * (1 - s)))).to(torch.bfloat16)
        zs.zero_fp8_quantize(du, *self.du8, *self.dut8)
        zs.zero_fp8_matmul(*self.du8, *self.upt8, self.dy, self.mm_ws)
        zs.zero_fp8_quantize(self.y, None, None, *self.yt8)
        zs.zero_fp8_matmul(*self.dut8, *self.yt8, dup, self.mm_ws)
        zs.zero_rmsnorm_backward(self.dy, self.h, self.params[slot][0], self.rstd, self.dx, dw_norm, self.rms_ws,
                                 dres=dout)
        return self.dx

    def update(self):
        """The global norm, the clipped gradients into the flat buffer, the step."""
        zs.zero_tensors_norm(self.grad_list, 1.0, self.stat, self.norm_ws)
        zs.zero_tensors_clip(self.grad_list, self.flat_list, 1.0, self.max_norm, self.stat)
        self.step.step([self.flat_grad])


def train(layer: Layer, x, residual, target, steps: int):
    """Mean squared error to `target`; (loss, gradient norm) of each step."""
    seen = []
    for _ in range(steps):
        slot = layer.step.read_state().cur
        err = layer.forward(x, residual, slot).float() - target.float()
        loss = err.square().mean()
        layer.backward((err * (2.0 / err.numel())).to(torch.bfloat16), slot)
        layer.update()
        if zs.read_matmul_error(layer.mm_ws):
            raise RuntimeError("a product gave up waiting: its output is undefined")
        seen.append((float(loss), zs.read_tensors_stat(layer.stat).norm))
    return seen


def main(steps: int = 30):
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens, d, ffn = 2048, 1024, 4096
    x, residual, target = (torch.randn(tokens, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    for i, (loss, norm) in enumerate(train(Layer(tokens, d, ffn), x, residual, target, steps)):
        print(f"step {i + 1:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main(*map(int, sys.argv[1:]))
