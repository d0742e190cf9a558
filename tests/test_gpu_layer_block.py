"""The example that runs the linear layer, its backward pass and the few-token
MoE layer together, against the same layers in 64 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "layer_block.py")
    spec = importlib.util.spec_from_file_location("layer_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def experts64(b, j):
    def of(w):
        q, s = w
        return q[j].float().to(F64) * s[j].to(F64).repeat_interleave(128, 0).repeat_interleave(128, 1)
    return of(b.w13), of(b.w2)


@pytest.mark.parametrize("tokens", [1, 5])
def test_block_and_its_graph(example, tokens):
    say(f"layer block {tokens} tokens")
    b = example.Block(hidden=512, intermediate=256, experts=8, top_k=2, tokens=tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn((tokens, 512), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out = b.step(x, r).clone()
    # each call from what it was given: the stream and the logits are rounded once, to bf16 and fp32
    pre = x.to(F64) @ b.wo.to(F64).t() + b.bo.to(F64)
    stream = pre + r.to(F64)
    size = x.to(F64).abs() @ b.wo.to(F64).abs().t() + b.bo.to(F64).abs() + r.to(F64).abs()
    assert ((b.stream.to(F64) - stream).abs() <= 2.0 ** -8 * stream.abs() + 2.0 ** -16 * size).all()
    s = b.stream.to(F64)
    logits = s @ b.router.to(F64).t()
    assert ((b.logits.to(F64) - logits).abs() <= 2.0 ** -16 * (s.abs() @ b.router.to(F64).abs().t())).all()
    top = torch.argsort(b.logits, dim=1, descending=True, stable=True)[:, :2]
    assert torch.equal(top.to(torch.int32), b.ids)
    w = torch.softmax(torch.gather(b.logits.to(F64), 1, top), 1)
    want, slack = s.clone(), s.abs()
    for t in range(tokens):
        for k in range(2):
            w13, w2 = experts64(b, int(b.ids[t, k]))
            z = s[t] @ w13.t()
            h = z[:256] / (1 + torch.exp(-z[:256])) * z[256:]
            want[t] += w[t, k] * (h @ w2.t())
            # h rounded to bf16, and fp32 sums below it: |z| sums enter through silu' <= 1.1
            c = s[t].abs() @ w13.abs().t()
            soft = 2.0 ** -8 * h.abs() + 2.0 ** -15 * (c[:256] * z[256:].abs() + c[256:] * z[:256].abs())
            slack[t] += w[t, k] * (2.0 ** 8 * soft @ w2.abs().t())
    assert ((out.to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -8 * slack).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(x, r)
    for k in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        b.out.fill_(float("nan"))
        graph.replay()
        replayed = b.out.clone()
        torch.cuda.synchronize()
        assert torch.equal(replayed, b.step(x, r)), k


def test_mlp_gradients_and_descent(example):
    """The gradients against those of the same network in 64 bits on the rounded
    weights, by their norms: six bf16 roundings of up to 2^-8 lie between the
    inputs and a gradient (hid, y, dy, dpre, dhid, the gradient itself), and
    y - target may be four times smaller than the rounded y."""
    say("layer block mlp")
    m = example.Mlp(width=64, hidden=256, rows=77)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((77, 64), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.roll(x, 1, 1)
    p = [t.to(torch.bfloat16).to(F64).requires_grad_() for t in (m.w1, m.w2)]
    p += [t.to(F64).requires_grad_() for t in (m.b1, m.b2)] + [x.to(F64).requires_grad_()]
    y = torch.nn.functional.gelu(p[4] @ p[0].t() + p[2]) @ p[1].t() + p[3] + p[4]
    loss = 0.5 * (y - target.to(F64)).square().sum()
    want = torch.autograd.grad(loss, p)
    got = m.gradients(x, target)
    assert abs(got.item() - loss.item()) <= 0.02 * loss.item()
    for name, a, b in zip(("w1", "w2", "b1", "b2", "x"), (m.dw1, m.dw2, m.db1, m.db2, m.dx), want):
        off = ((a.to(F64) - b).norm() / b.norm()).item()
        assert off <= 6 * 4 * 2.0 ** -8, (name, off)
    losses = [m.step(x, target, 1e-3).item() for _ in range(20)]
    assert losses[-1] < 0.8 * losses[0], losses
