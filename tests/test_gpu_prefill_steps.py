"""Training steps of the example one after another, the second with fewer segments
than the first: its gradients are those of a fresh object, whatever the first
step left behind the last segment."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say
from tests.test_gpu_prefill_block import BF16, example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_layout_that_shrinks(example):  # noqa: F811
    say("prefill block, training steps")
    t, h, e, k = 333, 256, 6, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    used, fresh = example.Training(h, e, k, t), example.Training(h, e, k, t)
    x, dy = rn(t, h).to(BF16), rn(t, h).to(BF16)
    ids, w = example.route(rn(t, e), k)
    used.forward(x, ids, w)
    used.backward(x, w, dy)
    before = int((used.m_indices >= 0).sum())
    few = torch.where(ids < 2, ids, torch.full_like(ids, -1))  # (most tokens' experts are on other devices)
    results = []
    for m in (used, fresh):
        y = m.forward(x, few, w)
        results.append([y.clone(), *(v.clone() for v in m.backward(x, w, dy)), *(m.expert_gradient(j) for j in range(e))])
    behind = int((used.m_indices >= 0).nonzero().max()) // 128 * 128 + 128
    assert int((used.m_indices >= 0).sum()) < before and (used.a[behind:] != 0).any()  # (earlier rows are still there)
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b), i
