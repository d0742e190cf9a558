"""Workspaces that the binding makes live until the library has launched: ctypes
lets other threads run during the call, and a block given back before it could be
another thread's tensor by then."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def calls(dg):
    ids = torch.zeros((4096, 8), dtype=torch.int32, device="cuda")
    rows, counts = torch.empty_like(ids), torch.empty(16, dtype=torch.int32, device="cuda")
    m_indices = torch.empty(dg.moe_sort_rows(4096, 8, 16), dtype=torch.int32, device="cuda")
    x, dw = torch.ones((4096, 512), dtype=torch.bfloat16, device="cuda"), torch.empty(512, device="cuda")
    return {
        "dg_moe_sort_contiguous": (4, dg.moe_sort_workspace(4096, 8, 16),
                                   lambda: dg.moe_sort_contiguous(ids, 16, m_indices, rows)),
        "dg_moe_sort_masked": (3, dg.moe_sort_workspace(4096, 8, 16), lambda: dg.moe_sort_masked(ids, 64, counts, rows)),
        "dg_rmsnorm_bf16_backward": (12, dg.rmsnorm_bf16_backward_workspace(4096, 512),
                                     lambda: dg.rmsnorm_bf16_backward(x, x, None, torch.ones(4096, device="cuda"), None, dw)),
    }


@pytest.mark.parametrize("name", ["dg_moe_sort_contiguous", "dg_moe_sort_masked", "dg_rmsnorm_bf16_backward"])
def test_workspace_is_held_during_the_call(dg, monkeypatch, name):
    place, need, call = calls(dg)[name]
    seen = []

    def instead(*args):  # (what another thread might do at this moment)
        given = args[place]
        taken = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(4)]
        seen.append(all(t.data_ptr() >= given + need or t.data_ptr() + need <= given for t in taken))
        return 0

    assert need > 0
    monkeypatch.setattr(dg._lib, name, instead)
    call()
    assert seen == [True]
