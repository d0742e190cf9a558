"""Gradients of the routing weights over long rows.  A thread adds 8 products to one
another and each such piece to its sum, which are 8 + ceil(H / 4096) roundings of
2^-24; a wave and the workgroup add 6 + 7 more: at most ceil(H / 4096) + 21 of the
products' sizes."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def check(dg, dy, o, rows):
    h = dy.shape[1]
    dw = torch.full(rows.shape, float("nan"), device="cuda")
    dg.moe_combine_bf16_backward(dy, o, rows, None, None, dw)
    for t in range(rows.shape[0]):
        for j in range(rows.shape[1]):
            p = dy[t].to(F64) * o[int(rows[t, j])].to(F64)
            off = (dw[t, j].to(F64) - p.sum()).abs() / p.abs().sum()
            assert off <= (-(-h // 4096) + 21) * 2.0 ** -24, (t, j, off.item() * 2 ** 24)


@pytest.mark.parametrize("k", [2, 11])
@pytest.mark.parametrize("h", [4096, 4104, 131072, 1 << 20])
def test_small_products_behind_large_ones(dg, h, k):
    """Each thread's first product is one, the others half an ulp of it: a chain over the row loses all of them."""
    say(f"routing weights' gradients h={h} k={k}")
    o = torch.full((k, h), 2.0 ** -24, device="cuda").to(BF16)
    o[:, 0:4096:8] = 1
    dy = torch.ones((2, h), dtype=BF16, device="cuda")
    check(dg, dy, o, torch.arange(k, device="cuda").to(torch.int32).repeat(2, 1).contiguous())


@pytest.mark.parametrize("h", [8200, 131072, 1 << 20])
def test_long_rows(dg, h):
    say(f"routing weights' gradients h={h}")
    g = torch.Generator(device="cuda").manual_seed(31)
    dy, o = (torch.randn((n, h), generator=g, device="cuda").to(BF16) for n in (3, 6))
    check(dg, dy, o, torch.tensor([[0, 5], [1, 3], [4, 2]], dtype=torch.int32, device="cuda"))
