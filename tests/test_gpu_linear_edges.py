"""The linear layer and its backward pass where values or addresses are large.

Tolerances as in tests/test_gpu_linear.py, whose bounds hold for every finite
value of the pre-activation."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say
from tests.test_gpu_linear import BF16, F64, slope64, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def check_backward(dg, dc, a, b, pre, act, what):
    """The three gradients against the formulas in 64 bits."""
    (m, n), k = dc.shape, a.shape[1]
    da, db = torch.full((m, k), float("nan"), dtype=BF16, device="cuda"), torch.full((n, k), float("nan"), dtype=BF16, device="cuda")
    dbias = torch.full((n,), float("nan"), device="cuda")
    dg.gemm_bf16_nt_epilogue_backward(dc, a, b, pre, act, da, db, dbias)
    torch.cuda.synchronize()
    a64, b64, dc64 = a.to(F64), b.to(F64), dc.to(F64)
    d = dc64 * slope64(pre.to(F64), act) if act != "none" else dc64
    assert torch.isfinite(d).all()
    q, r = 2.0 ** -8 + 2.0 ** -16, 2.0 ** -8
    ref = d @ b64
    worst(da, ref, q * (d.abs() @ b64.abs()) + 2.0 ** -18 * (dc64.abs() @ b64.abs()) + r * ref.abs(), what + " da")
    ref = d.t() @ a64
    worst(db, ref, q * (d.t().abs() @ a64.abs()) + 2.0 ** -18 * (dc64.t().abs() @ a64.abs()) + r * ref.abs(), what + " db")
    worst(dbias, d.sum(0), 2.0 ** -16 * d.abs().sum(0) + 2.0 ** -18 * dc64.abs().sum(0), what + " dbias")


# Rows whose distance passes what 32-bit byte offsets reach: in chunks of 16 rows (few of them) or 64 (64 x 131072),
# past half of it and past the whole, dc alone or pre too.
@pytest.mark.parametrize("m,n,ld,both", [(19, 33, (1 << 26) + 1, True), (19, 33, 143_200_001, True),
                                         (19, 40, 143_200_001, False), (64, 131_071, (1 << 24) + 1, False),
                                         (64, 131_071, 34_000_001, False), (64, 131_072, 34_000_008, False)])
def test_backward_of_rows_far_apart(dg, m, n, ld, both):
    say(f"linear backward rows far apart {m}x{n} ld={ld} both={both}")
    k = 16
    g = torch.Generator(device="cuda").manual_seed(23)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")

    def apart(t):  # the same rows, ld elements apart in a buffer of NaN
        buf = torch.full(((m - 1) * ld + n,), float("nan"), dtype=BF16, device="cuda")
        v = buf.as_strided((m, n), (ld, 1))
        v.copy_(t)
        return v

    dc, pre = apart(rn(m, n).to(BF16)), rn(m, n).to(BF16)
    if both:
        pre = apart(pre)
    check_backward(dg, dc, rn(m, k).to(BF16), (rn(n, k) / 4).to(BF16), pre, "silu", f"far apart {m}x{n} {ld}")
