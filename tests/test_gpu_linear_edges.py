"""The linear layer and its backward pass where values or addresses are large:
pre-activations up to bf16's largest value, rows any distance apart, views of
one row.

Tolerances as in tests/test_gpu_linear.py, whose bounds hold for every finite
value of the pre-activation: an activation's slope is 0 or 1 (or between) there
too."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say
from tests.test_gpu_linear import ACTS, BF16, F64, act64, slope64, worst

pytestmark = pytest.mark.gpu
LARGE = [1e2, 1e4, 1e9, 1e12, 1.3e13, 1e16, 1e19, 2e19, 1e25, 1e30, 3e38, 3.38e38]


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


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [40, 41])  # rows on 16-byte boundaries, and not
def test_backward_of_large_pre_activations(dg, act, n):
    say(f"linear backward large pre {act} n={n}")
    m, k = 50, 64
    g = torch.Generator(device="cuda").manual_seed(21)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    large = torch.tensor([s * v for v in LARGE for s in (1.0, -1.0)], device="cuda")
    pre = 2 * rn(m, n)
    pick = torch.rand((m, n), generator=g, device="cuda") < 0.5
    pre = torch.where(pick, large[torch.randint(0, len(large), (m, n), generator=g, device="cuda")], pre).to(BF16)
    assert torch.isfinite(pre.float()).all()
    check_backward(dg, rn(m, n).to(BF16), rn(m, k).to(BF16), (rn(n, k) / 8).to(BF16), pre, act, f"large pre {act} {n}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(5, 48), (5, 49), (80, 48), (80, 49)])
def test_forward_of_large_pre_activations(dg, act, m, n):
    """The bias brings the pre-activation up to 3.38e38; the products are of size 1."""
    say(f"linear forward large pre {act} {m}x{n}")
    k = 64
    g = torch.Generator(device="cuda").manual_seed(22)
    a, b = torch.randn((m, k), generator=g, device="cuda").to(BF16), (torch.randn((n, k), generator=g, device="cuda") / 8).to(BF16)
    bias = torch.zeros(n, device="cuda")
    bias[:2 * len(LARGE)] = torch.tensor([s * v for v in LARGE for s in (1.0, -1.0)], device="cuda")
    out, pre = torch.empty((m, n), device="cuda"), torch.empty((m, n), dtype=BF16, device="cuda")
    dg.gemm_bf16_nt_epilogue(a, b, out, bias, act, None, pre)
    z = a.to(F64) @ b.to(F64).t() + bias.to(F64)
    c = a.to(F64).abs() @ b.to(F64).abs().t() + bias.to(F64).abs()
    ref = act64(z, act)
    worst(out, ref, 1.2 * 2.0 ** -16 * c + 2.0 ** -20 * z.abs() + 2.0 ** -22 * ref.abs(), f"{act} {m}x{n}")
    worst(pre, z, 2.0 ** -16 * c + 2.0 ** -8 * z.abs(), f"{act} {m}x{n} pre")


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


@pytest.mark.parametrize("steps,step", [(3, 1), (4096, 4095), (2, 0)])
def test_one_row_of_a_longer_tensor(dg, steps, step):
    """x[:, -1] of a batch of one sequence: the stride of its one row is the
    whole sequence, and means nothing."""
    say(f"linear one row of {steps}")
    n, k = 264, 520
    g = torch.Generator(device="cuda").manual_seed(24)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, res = rn(1, steps, k).to(BF16)[:, step], rn(1, steps, n + 1).to(BF16)[:, step, :n]
    w = (rn(n, k) / k ** 0.5).to(BF16)
    out, pre = (torch.full((1, steps, n + 3), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    dg.gemm_bf16_nt_epilogue(x, w, out[:, step, :n], None, "silu", res, pre[:, step, :n])
    want, wpre = (torch.empty((1, n), dtype=BF16, device="cuda") for _ in range(2))
    dg.gemm_bf16_nt_epilogue(x.clone(), w, want, None, "silu", res.clone(), wpre)
    assert torch.equal(out[:, step, :n], want) and torch.equal(pre[:, step, :n], wpre)
    assert torch.isnan(out[:, step, n:].float()).all()
    check_backward(dg, res, x, w, pre[:, step, :n], "silu", f"one row of {steps}")
