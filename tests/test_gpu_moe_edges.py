"""Routing of the few-token MoE layer where sigmoids leave fp32's range, and its
layers wider than 16 columns per compute unit (the 32-column form of the down
kernel).  Tolerances as in tests/test_gpu_moe_few_tokens.py."""
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


@pytest.mark.parametrize("t,e,k,h,i", [(1, 4, 2, 4224, 128), (1, 3, 3, 7168, 1152), (5, 6, 4, 7168, 384),
                                       (16, 5, 2, 4224, 1664), (17, 4, 3, 4224, 384), (40, 20, 4, 7168, 128),
                                       (64, 3, 2, 4352, 256)])
@pytest.mark.parametrize("fp8", [True, False])
def test_wide_layers(dg, t, e, k, h, i, fp8):
    say(f"moe wide t={t} e={e} k={k} h={h} i={i} fp8={fp8}")
    assert h > 16 * torch.cuda.get_device_properties(0).multi_processor_count, "not the 32-column form"
    d = make(t, e, k, h, i, fp8, 200 + t + h)
    out, ids, w = call(dg, d, fp8, t, k, scale=0.75)
    rid, rw = topk_reference(d["logits"], k, "softmax", True, 0.75)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.abs(w.cpu().numpy() - rw).max() <= 2.0 ** -20
    ref, bound = reference(d, rid, w.cpu(), True)
    check(out, ref, bound, f"wide {t} {e} {k} {h} {i} {fp8}")
    again = call(dg, d, fp8, t, k, scale=0.75)[0]
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not deterministic"


@pytest.mark.parametrize("t", [9, 30])
@pytest.mark.parametrize("fp8", [True, False])
def test_wide_layers_with_given_ids(dg, t, fp8):
    e, k, h, i = 6, 4, 4224, 256
    say(f"moe wide given ids t={t} fp8={fp8}")
    assert h > 16 * torch.cuda.get_device_properties(0).multi_processor_count, "not the 32-column form"
    d = make(t, e, k, h, i, fp8, 41)
    g = torch.Generator().manual_seed(42)
    ids = torch.randint(-1, e + 2, (t, k), generator=g).to(torch.int32)
    ids[0] = -1                                                  # a token without experts
    ids[1] = torch.tensor([2, 2, 2, 2])
    ids[3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 5])
    w = torch.randn(t, k, generator=g)
    for residual in (True, False):
        out, _, _ = call(dg, d, fp8, t, k, ids=ids, weights=w, residual=residual)
        ref, bound = reference(d, ids, w, residual)
        check(out[1:], ref[1:], bound[1:], f"wide given ids residual={residual}")
        want = d["residual"][0].float() if residual else torch.zeros(h)
        assert torch.equal(out[0].float().cpu(), want)
