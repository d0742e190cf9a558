"""Dispatch of FP8 rows with packed UE8M0 scales where the padding rows become
zeros: bit for bit, the words of a row's last groups partly padding."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say
from tests.test_gpu_moe_rows import DISPATCH, FP8, dg, routing, sorted_rows, spread64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,k,e,h", sorted({(t, k, e, max(128, h // 128 * 128)) for t, k, e, h in DISPATCH}
                                           | {(70, 2, 5, 128), (70, 2, 5, 640), (9, 3, 4, 33408)}))
def test_padding_of_zeros_with_packed_scales(dg, t, k, e, h):  # noqa: F811
    say(f"dispatch padding ue8m0 {t}x{k} of {e} h={h}")
    ids = routing(t, k, e, 7, "holes")
    rows, m_indices, m = sorted_rows(dg, ids, e, False)
    used = (m_indices.view(-1, 128) >= 0).any(1).repeat_interleave(128)
    g = torch.Generator(device="cuda").manual_seed(8)
    words = (h + 511) // 512
    x = torch.randint(0, 256, (t, h), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(-2 ** 31, 2 ** 31 - 1, (t, words), generator=g, device="cuda", dtype=torch.int32)
    a = torch.full((m, h), 9, dtype=torch.uint8, device="cuda")
    sa = torch.full((m, words), 9, dtype=torch.int32, device="cuda")
    dg.moe_dispatch_fp8((x.view(FP8), s), rows, (a.view(FP8), sa), m_indices)
    for got, src in ((a, x), (sa, s)):
        assert torch.equal(got[used], spread64(src, rows, m, 0)[used]) and (got[~used] == 9).all()
