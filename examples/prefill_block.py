"""A mixture-of-experts block for many tokens, its training step, and an INT8 layer.

    python examples/prefill_block.py          (one MI355X)

`Prefill` is what a prompt does after attention, in FP8: the norm adds the
attention's output to the residual stream and writes the experts' operand, the
tokens are sorted by expert into the contiguous layout, the two grouped GEMMs
run (SwiGLU and re-quantisation inside the first), and the experts' outputs come
back weighted, added to the stream -- seven library calls, every buffer made
once.  `Training` is the same path in BF16 with one linear layer per expert, and
its gradients.  `Int8Mlp` is a dense two-layer network on INT8 weights.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_grouped_gemm_x128_amd as dg  # noqa: E402

BF16, F32, I32, FP8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def route(logits, top_k):
    """Experts int32 [T,k] and softmax weights fp32 [T,k] of router logits [T,E]."""
    top, ids = torch.topk(logits, top_k, dim=1)
    return ids.to(I32), torch.softmax(top, 1)


class Prefill:
    """Norm, experts on FP8 weights and the weighted sum for up to `tokens` tokens."""

    def __init__(self, hidden=1024, intermediate=512, experts=8, top_k=2, tokens=300, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device=device) / math.sqrt(s[-1])
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=device)
        h, i, e, t = hidden, intermediate, experts, tokens
        self.experts, self.norm = e, (1 + 0.1 * torch.randn(h, generator=g, device=device)).to(BF16)
        self.w13, self.s13 = self._quantise(rn(e, 2 * i, h))
        self.w2, self.s2 = self._quantise(rn(e, h, i))
        m = dg.moe_sort_rows(t, top_k, e)
        self.q, self.s = new(t, h, dtype=FP8), new(t, h // 128, dtype=F32)
        self.m_indices, self.rows = new(m, dtype=I32), new(t, top_k, dtype=I32)
        self.a, self.sa = new(m, h, dtype=FP8), new(m, h // 128, dtype=F32)
        self.hid, self.shid = new(m, i, dtype=FP8), new(m, i // 128, dtype=F32)
        self.o, self.out = new(m, h), new(t, h)
        self.workspace = new(max(1, dg.moe_sort_workspace(t, top_k, e)), dtype=torch.uint8)

    @staticmethod
    def _quantise(w):
        q, s = zip(*(dg.quantize_fp8_128x128(x.contiguous()) for x in w))
        return torch.stack([x.view(torch.uint8) for x in q]).view(FP8), torch.stack(s)

    def step(self, attended, stream, ids, weights):
        """attended bf16 [T,H] is added to stream bf16 [T,H] in place; returns the stream after the experts."""
        dg.rmsnorm_quantize_fp8_1x128(attended, self.norm, self.q, self.s, residual=stream, sum_out=stream)
        dg.moe_sort_contiguous(ids, self.experts, self.m_indices, self.rows, workspace=self.workspace)
        dg.moe_dispatch_fp8((self.q, self.s), self.rows, (self.a, self.sa))
        dg.dg_grouped_fp8_contiguous_swiglu(self.a, self.sa, self.w13, self.s13, self.hid, self.shid, self.m_indices)
        dg.dg_grouped_fp8_contiguous(self.hid, self.shid, self.w2, self.s2, self.o, self.m_indices)
        return dg.moe_combine_bf16(self.o, self.rows, self.out, weights, stream)


class Training:
    """x + sum_j weights_j expert_j(norm(x)) with one linear layer per expert, forward and backward in BF16."""

    def __init__(self, hidden=512, experts=6, top_k=2, tokens=333, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        h, e, t = hidden, experts, tokens
        self.experts = e
        self.norm = 1 + 0.1 * torch.randn(h, generator=g, device=device)
        self.w = (torch.randn((e, h, h), generator=g, device=device) / math.sqrt(h)).to(BF16)
        self.wt = self.w.transpose(1, 2).contiguous()
        m = dg.moe_sort_rows(t, top_k, e)
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=device)
        self.m_indices, self.rows = new(m, dtype=I32), new(t, top_k, dtype=I32)
        self.n, self.y, self.dn, self.dx = (new(t, h) for _ in range(4))
        # rows behind the last segment keep what an earlier step with more segments left there: products of whole
        # buffers leave them out by m_indices (as the grouped GEMMs and expert_gradient do)
        self.a, self.o, self.do, self.da = (torch.zeros((m, h), dtype=BF16, device=device) for _ in range(4))
        self.rstd, self.dnorm, self.dweights = new(t, dtype=F32), new(h, dtype=F32), new(t, top_k, dtype=F32)

    def forward(self, x, ids, weights):
        dg.rmsnorm_bf16(x, self.norm, self.n, rstd=self.rstd)
        dg.moe_sort_contiguous(ids, self.experts, self.m_indices, self.rows)
        dg.moe_dispatch_bf16(self.n, self.rows, self.a, self.m_indices)
        dg.dg_grouped_bf16_contiguous(self.a, self.w, self.o, self.m_indices)
        return dg.moe_combine_bf16(self.o, self.rows, self.y, weights, x)

    def backward(self, x, weights, dy):
        """From dy bf16 [T,H]: the gradients of x, the norm's weight, the routing weights, and (as pairs of operands
        `do`, `a` in the contiguous layout, zeros in its segments' padding) those of the experts' weights."""
        dg.moe_combine_bf16_backward(dy, self.o, self.rows, weights, self.do, self.dweights, self.m_indices)
        dg.dg_grouped_bf16_contiguous(self.do, self.wt, self.da, self.m_indices)
        dg.moe_dispatch_bf16_backward(self.da, self.rows, self.dn)
        dg.rmsnorm_bf16_backward(self.dn, x, self.norm, self.rstd, self.dx, self.dnorm, dsum=dy)
        return self.dx, self.dnorm, self.dweights

    def expert_gradient(self, e):
        """dW of expert e: do^T a over its segment."""
        at = (self.m_indices == e).nonzero()[:, 0]
        last = int(at[-1]) // 128 * 128 + 128 if at.numel() else 0
        first = int(at[0]) if at.numel() else 0
        return self.do[first:last].float().t() @ self.a[first:last].float()


class Int8Mlp:
    """stream + W2 gelu(W1 norm(stream) + b1) + b2 on INT8 weights, activations quantised per token."""

    def __init__(self, width=1024, hidden=2816, tokens=200, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.norm = torch.ones(width, device=device)
        self.w1 = dg.quantize_int8_rows(torch.randn((hidden, width), generator=g, device=device) / math.sqrt(width))
        self.w2 = dg.quantize_int8_rows(torch.randn((width, hidden), generator=g, device=device) / math.sqrt(hidden))
        self.b1, self.b2 = (0.1 * torch.randn(n, generator=g, device=device) for n in (hidden, width))
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device=device)
        self.x = new(tokens, width, dtype=torch.int8), new(tokens, dtype=F32)
        self.h = new(tokens, hidden, dtype=BF16)
        self.hq = new(tokens, hidden, dtype=torch.int8), new(tokens, dtype=F32)
        self.out = new(tokens, width, dtype=BF16)

    def step(self, stream):
        dg.rmsnorm_quantize_int8(stream, self.norm, *self.x)
        dg.gemm_int8_nt_epilogue(self.x, self.w1, self.h, self.b1, "gelu")
        dg.dg_quantize_int8_rows(self.h, *self.hq)
        return dg.gemm_int8_nt_epilogue(self.hq, self.w2, self.out, self.b2, "none", stream)


def main():
    t, h, e, k = 4096, 4096, 32, 4
    block = Prefill(h, 1536, e, k, t)
    x, stream = (torch.randn((t, h), device="cuda").to(BF16) for _ in range(2))
    ids, weights = route(torch.randn((t, e), device="cuda"), k)
    mlp = Int8Mlp(h, 11008, t)
    train = Training(1024, 8, 2, 2048)
    tx, dy = (torch.randn((2048, 1024), device="cuda").to(BF16) for _ in range(2))
    tids, tw = route(torch.randn((2048, 8), device="cuda"), 2)

    def training():
        train.forward(tx, tids, tw)
        train.backward(tx, tw, dy)

    for name, f in (("FP8 experts, 4096 tokens", lambda: block.step(x, stream, ids, weights)),
                    ("INT8 layers, 4096 tokens", lambda: mlp.step(stream)),
                    ("BF16 experts forward and backward, 2048 tokens", training)):
        f()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            f()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {1e3 * start.elapsed_time(end) / 20:.1f} us")


if __name__ == "__main__":
    main()
