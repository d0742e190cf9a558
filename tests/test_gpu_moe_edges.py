"""Routing of the few-token MoE layer where sigmoids leave fp32's range.
Tolerances as in tests/test_gpu_moe_few_tokens.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.parity import say
from tests.test_gpu_moe_few_tokens import call, check, make, reference, topk_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def test_renormalised_sigmoids_below_fp32(dg):
    """Weights are quotients of sigmoids: where all of them are below fp32's
    smallest values the quotients are not.  (Below -745 the sigmoids are zero in
    64 bits as well: a mask, weight 0.)"""
    t, e, k, h, i = 10, 20, 4, 128, 128
    say("moe small sigmoids")
    d = make(t, e, k, h, i, True, 31)
    base = [0.0, -15.0, -19.9, -20.1, -60.0, -88.0, -95.0, -104.0, -300.0, -700.0]
    l = torch.stack([b + d["logits"][r] for r, b in enumerate(base)])
    l[4, 7:] = float("-inf")
    l[5, :] = -100.0                      # all alike: 1 / k
    l[8, 3:] = -1e30                      # three experts and masks
    d["logits"] = l
    out, ids, w = call(dg, d, True, t, k, scoring="sigmoid")
    rid, rw = topk_reference(l, k, "sigmoid", True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # an exponential of fp32 (an argument of up to 8, rounded to 2^-21, and the result to 2^-23), a sum and a quotient
    assert np.abs(w.cpu().numpy() - rw).max() <= 2.0 ** -19
    assert np.allclose(w.sum(1).cpu().numpy(), 1, atol=2.0 ** -20)
    ref, bound = reference(d, rid, w.cpu(), True)
    check(out, ref, bound, "small sigmoids")
