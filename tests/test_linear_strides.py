"""Row strides that the Python entry points hand on (no GPU: the helper takes
the device to expect, -1 for the host)."""
from __future__ import annotations

import pytest
import torch

import moe_grouped_gemm_x128_amd as dg


def test_one_row_has_no_stride():
    x = torch.empty(1, 4096, 520)
    assert dg._ld(x[:, -1], -1, "x") == 520
    assert dg._ld(x[0, :1].expand(1, 520), -1, "x") == 520
    assert dg._ld(torch.empty(3, 527)[1:2, :520], -1, "x") == 520


def test_rows_keep_their_stride():
    assert dg._ld(torch.empty(3, 528)[:, :520], -1, "x") == 528
    assert dg._ld(torch.empty(3, 520), -1, "x") == 520
    for bad in (torch.empty(1, 520).expand(3, 520), torch.empty(520, 3).t(), torch.empty(3, 520)[:, ::2]):
        with pytest.raises(ValueError):
            dg._ld(bad, -1, "x")
