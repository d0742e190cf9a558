"""The linear layer, its backward pass and the few-token MoE layer together.

    python examples/layer_block.py          (one MI355X)

`Block` is what a generation step does after attention, for a handful of
tokens: the output projection added to the residual stream, the router's logits
(fp32), and the mixture of experts with its own residual -- three library calls
and four kernels.  Every buffer is made once, so a step can be captured in a
graph.  `Mlp` is a training step of a two-layer network: forward calls that keep
the pre-activations, and their backward passes.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_x128_amd as dg  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Block:
    """Projection, router and experts for up to 64 tokens, on FP8 weights."""

    def __init__(self, hidden=1024, intermediate=512, experts=8, top_k=2, tokens=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device=device) / math.sqrt(s[-1])
        h, i, e, t = hidden, intermediate, experts, tokens
        self.wo, self.bo = rn(h, h).to(BF16), 0.1 * torch.randn(h, generator=g, device=device)
        self.router = rn(e, h).to(BF16)
        self.w13 = self._quantise(rn(e, 2 * i, h))
        self.w2 = self._quantise(rn(e, h, i))
        self.stream, self.out = (torch.empty((t, h), dtype=BF16, device=device) for _ in range(2))
        self.logits = torch.empty((t, e), dtype=F32, device=device)
        self.ids = torch.empty((t, top_k), dtype=torch.int32, device=device)
        self.weights = torch.empty((t, top_k), dtype=F32, device=device)
        self.workspace = torch.empty(t * top_k * i, dtype=BF16, device=device)

    @staticmethod
    def _quantise(w):
        q, s = zip(*(dg.quantize_fp8_128x128(x.contiguous()) for x in w))
        return torch.stack([x.view(torch.uint8) for x in q]).view(torch.float8_e4m3fn), torch.stack(s)

    def step(self, attended, residual):
        """attended, residual bf16 [T,H] -> the residual stream after the block."""
        dg.gemm_bf16_nt_epilogue(attended, self.wo, self.stream, self.bo, "none", residual)
        dg.gemm_bf16_nt_epilogue(self.stream, self.router, self.logits)
        return dg.moe_few_tokens_fp8(self.stream, self.w13, self.w2, self.out, self.ids, self.weights,
                                     logits=self.logits, residual=self.stream, workspace=self.workspace)


class Mlp:
    """x + W2 gelu(W1 x + b1) + b2 with fp32 master weights and plain gradient descent."""

    def __init__(self, width=512, hidden=2048, rows=777, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.w1 = torch.randn((hidden, width), generator=g, device=device) / math.sqrt(width)
        self.w2 = torch.randn((width, hidden), generator=g, device=device) / math.sqrt(hidden)
        self.b1, self.b2 = torch.zeros(hidden, device=device), torch.zeros(width, device=device)
        new = lambda *s: torch.empty(s, dtype=BF16, device=device)
        self.hid, self.pre, self.dhid = new(rows, hidden), new(rows, hidden), new(rows, hidden)
        self.y, self.dx = new(rows, width), new(rows, width)
        self.dw1, self.dw2 = new(hidden, width), new(width, hidden)
        self.db1, self.db2 = torch.empty_like(self.b1), torch.empty_like(self.b2)
        need = max(dg.gemm_bf16_nt_epilogue_backward_workspace(rows, n) for n in (hidden, width))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)

    def gradients(self, x, target):
        """Loss and (in dw1, db1, dw2, db2, dx) the gradients of sum((y - target)^2) / 2."""
        w1, w2 = self.w1.to(BF16), self.w2.to(BF16)
        dg.gemm_bf16_nt_epilogue(x, w1, self.hid, self.b1, "gelu", None, self.pre)
        dg.gemm_bf16_nt_epilogue(self.hid, w2, self.y, self.b2, "none", x)
        diff = self.y.float() - target.float()
        dy = diff.to(BF16)
        dg.gemm_bf16_nt_epilogue_backward(dy, self.hid, w2, None, "none", self.dhid, self.dw2, self.db2,
                                          self.workspace)
        dg.gemm_bf16_nt_epilogue_backward(self.dhid, x, w1, self.pre, "gelu", self.dx, self.dw1, self.db1,
                                          self.workspace)
        self.dx += dy  # the residual's share
        return 0.5 * diff.square().sum()

    def step(self, x, target, rate):
        loss = self.gradients(x, target)
        for w, d in ((self.w1, self.dw1), (self.w2, self.dw2), (self.b1, self.db1), (self.b2, self.db2)):
            w -= rate * d.float()
        return loss


def main():
    block = Block(hidden=4096, intermediate=1536, experts=16, top_k=4, tokens=8)
    x, r = (torch.randn((8, 4096), device="cuda").to(BF16) for _ in range(2))
    block.step(x, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(x, r)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"block of 8 tokens: {1e3 * start.elapsed_time(end) / 100:.1f} us a step")

    mlp = Mlp()
    x = torch.randn((777, 512), device="cuda").to(BF16)
    target = torch.roll(x, 1, 1)
    for step in range(31):
        loss = mlp.step(x, target, 5e-6)
        if step % 10 == 0:
            print(f"training step {step}: loss {loss.item():.4g}")


if __name__ == "__main__":
    main()
