"""The example that runs the norm, the sorted tokens, the grouped GEMMs and the
INT8 layer together, against the same layers in 64 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prefill_block.py")
    spec = importlib.util.spec_from_file_location("prefill_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def values(q, s, rows=1):
    return q.float().to(F64) * s.to(F64).repeat_interleave(rows, 0).repeat_interleave(128, 1)


def within(got, want, bound, what):
    bad = ~((got.to(F64) - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


def inputs(t, h, e, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r = (torch.randn((t, h), generator=g, device="cuda").to(BF16) for _ in range(2))
    return x, r, torch.randn((t, e), generator=g, device="cuda")


@pytest.mark.parametrize("tokens", [1, 70, 300])
def test_prefill_block_and_its_graph(example, tokens):
    """Each step from what it was given.  The grouped GEMM's FP8 sums are within 2^-15 of the products' sizes, SwiGLU
    sees its two projections rounded to bf16 (2^-8 each, through slopes of at most 1.1), and e4m3 adds 2^-4 and half
    its smallest step, 2^-10 of the scale."""
    say(f"prefill block {tokens} tokens")
    h, i, e, k = 512, 256, 8, 2
    b = example.Prefill(h, i, e, k, tokens)
    x, stream, logits = inputs(tokens, h, e, k, 1)
    ids, w = example.route(logits, k)
    before = stream.clone()
    out = b.step(x, stream, ids, w).clone()
    z = x.to(F64) + before.to(F64)
    within(stream, z, (2.0 ** -8 + 2.0 ** -24) * z.abs(), "stream")
    y = z / torch.sqrt(z.square().mean(1, keepdim=True) + 1e-6) * b.norm.to(F64)
    se = b.s.to(F64).repeat_interleave(128, 1)
    within(values(b.q, b.s), y, (2.0 ** -4 + 2.0 ** -15) * y.abs() + 2.0 ** -10 * se, "norm")
    xq, want, size = values(b.q, b.s), stream.to(F64), stream.to(F64).abs()
    for t in range(tokens):
        for j in range(k):
            ex, row = int(ids[t, j]), int(b.rows[t, j])
            assert b.m_indices[row] == ex
            w13, w2 = values(b.w13[ex], b.s13[ex], 128), values(b.w2[ex], b.s2[ex], 128)
            p = xq[t] @ w13.t()
            c = xq[t].abs() @ w13.abs().t()
            off = 2.0 ** -15 * c + 2.0 ** -8 * p.abs()
            gate, up = p[:i], p[i:]
            hid = gate / (1 + torch.exp(-gate)) * up
            soft = 1.1 * (off[:i] * up.abs() + off[i:] * gate.abs() + off[:i] * off[i:])
            got = values(b.hid[row:row + 1], b.shid[row:row + 1])[0]
            sh = b.shid[row].to(F64).repeat_interleave(128)
            within(got, hid, 1.07 * soft + (2.0 ** -4 + 2.0 ** -15) * hid.abs() + 2.0 ** -10 * sh, "hidden")
            o = got @ w2.t()
            within(b.o[row], o, 2.0 ** -15 * (got.abs() @ w2.abs().t()) + 2.0 ** -8 * o.abs(), "expert")
            term = w[t, j].to(F64) * b.o[row].to(F64)
            want[t] += term
            size[t] += term.abs()
    within(out, want, 2.0 ** -8 * want.abs() + 2.0 ** -19 * size, "out")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(x, stream, ids, w)
    for n in range(3):
        nx, ns, nl = inputs(tokens, h, e, k, 10 + n)
        nids, nw = example.route(nl, k)
        x.copy_(nx), stream.copy_(ns), ids.copy_(nids), w.copy_(nw)
        b.out.fill_(float("nan"))
        graph.replay()
        replayed = b.out.clone()
        torch.cuda.synchronize()
        stream.copy_(ns)
        assert torch.equal(replayed, b.step(x, stream, ids, w)), n


def test_training_gradients(example):
    """By norms, against autograd in 64 bits on the same rounded weights: between inputs and a gradient lie at most six
    roundings to bf16 (n, o or do, da, dn, the result, and y's terms), 2^-8 each at most of values that are not
    smaller than a fourth of the result's."""
    say("prefill block training")
    t, h, e, k = 333, 256, 6, 2
    m = example.Training(h, e, k, t)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn((t, h), generator=g, device="cuda").to(BF16) for _ in range(2))
    ids, w = example.route(torch.randn((t, e), generator=g, device="cuda"), k)
    ids[::7, 1] = -1  # (an expert on another device)
    y = m.forward(x, ids, w)
    dx, dnorm, dw = m.backward(x, w, dy)
    p = [v.to(F64).requires_grad_() for v in (x, m.norm, w, m.w)]
    n = p[0] / torch.sqrt(p[0].square().mean(1, keepdim=True) + 1e-6) * p[1]
    ok = (ids >= 0).to(F64)
    # (a product for every expert, the chosen ones picked: one expert's weights at a time)
    every = torch.stack([n @ p[3][j].t() for j in range(e)], 1)
    picked = torch.gather(every, 1, ids.clamp(min=0).long()[:, :, None].expand(-1, -1, h))
    want = p[0] + ((p[2] * ok)[:, :, None] * picked).sum(1)
    grads = torch.autograd.grad((want * dy.to(F64)).sum(), p)
    assert ((y.to(F64) - want).norm() / want.norm()) <= 3 * 2.0 ** -8
    for name, a, b in (("x", dx, grads[0]), ("norm", dnorm, grads[1]), ("routing", dw * ok, grads[2])):
        off = ((a.to(F64) - b).norm() / b.norm()).item()
        assert off <= 6 * 4 * 2.0 ** -8, (name, off)
    for j in range(e):
        off = ((m.expert_gradient(j).to(F64) - grads[3][j]).norm() / grads[3][j].norm()).item()
        assert off <= 6 * 4 * 2.0 ** -8, (j, off)


@pytest.mark.parametrize("tokens", [3, 200])
def test_int8_layers(example, tokens):
    """Each layer from what it was given: exact sums, three fp32 roundings and the bf16 one."""
    say(f"int8 layers {tokens} tokens")
    m = example.Int8Mlp(512, 768, tokens)
    stream = inputs(tokens, 512, 1, 1, 5)[0]
    out = m.step(stream)
    f = lambda v: v[0].to(F64) * v[1].to(F64)[:, None]
    z = stream.to(F64)
    y = z / torch.sqrt(z.square().mean(1, keepdim=True) + 1e-6)
    within(f(m.x), y, 0.5 * m.x[1].to(F64)[:, None] + 2.0 ** -15 * y.abs(), "norm")
    pre = f(m.x) @ f(m.w1).t() + m.b1.to(F64)
    hid = torch.nn.functional.gelu(pre)
    within(m.h, hid, 2.0 ** -8 * hid.abs() + 2.0 ** -19 * (pre.abs() + m.b1.to(F64).abs()), "hidden")
    within(f(m.hq), m.h.to(F64), 0.5 * m.hq[1].to(F64)[:, None] + 2.0 ** -22 * m.h.to(F64).abs(), "codes")
    p = f(m.hq) @ f(m.w2).t()
    want = p + m.b2.to(F64) + z
    within(out, want, 2.0 ** -8 * want.abs() + 2.0 ** -20 * (p.abs() + m.b2.to(F64).abs() + z.abs()), "out")
