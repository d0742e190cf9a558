"""The norm's 8-bit outputs against the quantisers' on the same y.  The factor r
comes from the call itself and the header fixes the order of y's products, so y is
two fp32 products of known operands: INT8 and packed UE8M0 outputs are compared
bit for bit, FP8 with fp32 scales within the margin that the header gives (2^-20)
of 64 bits."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say
from tests.test_gpu_norm import BF16, F32, F64, FP8, dg, inputs  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS = [(1, 7168), (5, 128), (37, 2048), (700, 256), (64, 384), (9, 4224), (3, 8320), (2, 16384), (600, 1024)]
KINDS = [(True, BF16), (False, F32), (True, None)]


def normed(call, x, r, w):
    """z, the call's factor (as a column) and the weight, in fp32."""
    rstd = torch.empty(x.shape[0], device="cuda")
    call(rstd)
    z = x.float() if r is None else x.float() + r.float()
    return z, rstd[:, None], torch.ones(x.shape[1], device="cuda") if w is None else w.float()


@pytest.mark.parametrize("t,h", ROWS + [(3, 1), (4, 5), (17, 1000), (333, 2111), (2, 16383)])
@pytest.mark.parametrize("residual,weight", KINDS)
def test_int8_is_the_quantiser_s(dg, t, h, residual, weight):  # noqa: F811
    say(f"norm int8 rule {t}x{h}")
    x, r, w = inputs(t, h, residual, weight, 22)
    q, s = torch.zeros((t, h), dtype=torch.int8, device="cuda"), torch.zeros(t, device="cuda")
    z, rs, wf = normed(lambda rstd: dg.rmsnorm_quantize_int8(x, w, q, s, 1e-6, r, None, rstd), x, r, w)
    q2, s2 = dg.quantize_int8_rows(z * wf * rs)
    assert torch.equal(s, s2), int((s != s2).sum())
    assert torch.equal(q, q2), int((q != q2).sum())


@pytest.mark.parametrize("exponent", [-98, -60, -45, -30, 30, 90])
def test_int8_over_the_range(dg, exponent):  # noqa: F811
    """Weights that take the scales to where 1 / s leaves the ordinary range."""
    say(f"norm int8 rule 2^{exponent}")
    t, h = 40, 1024
    x, _, w = inputs(t, h, False, F32, 23)
    w = w * 2.0 ** exponent
    q, s = torch.zeros((t, h), dtype=torch.int8, device="cuda"), torch.zeros(t, device="cuda")
    z, rs, wf = normed(lambda rstd: dg.rmsnorm_quantize_int8(x, w, q, s, 0.0, None, None, rstd), x, None, w)
    q2, s2 = dg.quantize_int8_rows(z * wf * rs)
    assert torch.equal(s, s2) and torch.equal(q, q2)


@pytest.mark.parametrize("exponent", [-110, 122])
@pytest.mark.parametrize("h", [384, 1024, 9088])
def test_int8_where_the_products_leave_the_range(dg, h, exponent):  # noqa: F811
    """Factors near 2^-40 or 2^40 that the weights undo: the order is (z r) w here."""
    say(f"norm int8 rule, products 2^{exponent}, h={h}")
    t = 7
    x, _, w = inputs(t, h, False, F32, 24)
    sign = 1 if exponent > 0 else -1
    x, w = (x.float() * 2.0 ** (40 * sign)).to(BF16), w * 2.0 ** (exponent - 40 * sign)
    q, s = torch.zeros((t, h), dtype=torch.int8, device="cuda"), torch.zeros(t, device="cuda")
    z, rs, wf = normed(lambda rstd: dg.rmsnorm_quantize_int8(x, w, q, s, 0.0, None, None, rstd), x, None, w)
    q2, s2 = dg.quantize_int8_rows(z * rs * wf)
    assert torch.equal(s, s2) and torch.equal(q, q2)


@pytest.mark.parametrize("t,h", ROWS)
@pytest.mark.parametrize("residual,weight", KINDS)
def test_packed_fp8_is_the_quantiser_s(dg, t, h, residual, weight):  # noqa: F811
    say(f"norm ue8m0 rule {t}x{h}")
    x, r, w = inputs(t, h, residual, weight, 21)
    q, q2 = (torch.zeros((t, h), dtype=torch.uint8, device="cuda") for _ in range(2))
    s, s2 = (torch.zeros((t, (h + 511) // 512), dtype=torch.int32, device="cuda") for _ in range(2))
    z, rs, wf = normed(lambda rstd: dg.rmsnorm_quantize_fp8_1x128(x, w, q, s, 1e-6, r, None, rstd), x, r, w)
    dg.dg_quantize_fp8_1x128_ue8m0(z * rs * wf, q2, s2)
    assert torch.equal(s, s2) and torch.equal(q, q2)


def test_packed_fp8_next_to_the_least_scale(dg):  # noqa: F811
    """Around amax = 448 2^-127 the quotient is subnormal and is rounded before its power is taken.  Rows of ones:
    y is the weight."""
    say("norm ue8m0 least scale")
    h = 128
    amax = torch.tensor(448 * 2.0 ** -127, device="cuda").view(torch.int32)
    x = torch.ones((1, h), dtype=BF16, device="cuda")
    for step in range(-20, 21):
        w = torch.full((h,), 2.0 ** -140, device="cuda")
        w[5] = (amax + step).view(F32)
        q, q2 = (torch.zeros((1, h), dtype=torch.uint8, device="cuda") for _ in range(2))
        s, s2 = (torch.zeros((1, 1), dtype=torch.int32, device="cuda") for _ in range(2))
        dg.rmsnorm_quantize_fp8_1x128(x, w, q, s, 0.0)
        dg.dg_quantize_fp8_1x128_ue8m0(w[None].contiguous(), q2, s2)
        assert torch.equal(s, s2) and torch.equal(q, q2), step


# Against 64 bits: y carries 2 roundings and z one, amax the same, s two (FP8: a product with 1 / 448), its reciprocal
# one (FP8: an ulp, two) and the code's product one; r is the same in y and amax.  11 roundings of 2^-24 < 2^-20.
@pytest.mark.parametrize("t,h", ROWS)
@pytest.mark.parametrize("residual,weight", KINDS)
def test_codes_differ_from_64_bits_at_midpoints_alone(dg, t, h, residual, weight):  # noqa: F811
    say(f"norm codes against 64 bits {t}x{h}")
    x, r, w = inputs(t, h, residual, weight, 25)
    z = x.to(F64) + (0 if r is None else r.to(F64))
    y = z / torch.sqrt(z.square().mean(1, keepdim=True) + 1e-6) * (1 if w is None else w.to(F64))
    q, s = torch.zeros((t, h), dtype=torch.int8, device="cuda"), torch.zeros(t, device="cuda")
    dg.rmsnorm_quantize_int8(x, w, q, s, 1e-6, r)
    v = y / (y.abs().amax(1, keepdim=True) / 127)
    assert ((q.to(F64) - v).abs() <= 0.5 + 2.0 ** -20 * v.abs()).all()
    f, fs = torch.zeros((t, h), dtype=FP8, device="cuda"), torch.zeros((t, h // 128), device="cuda")
    dg.rmsnorm_quantize_fp8_1x128(x, w, f, fs, 1e-6, r)
    v = y / (y.view(t, -1, 128).abs().amax(2) / 448).repeat_interleave(128, 1)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    assert ((f.float().to(F64) - v).abs() <= 0.5 * step + 2.0 ** -20 * v.abs()).all()


@pytest.mark.parametrize("h", [5, 128, 300, 2111, 4096, 9000])
def test_bf16_rows_that_have_no_norm(dg, h):  # noqa: F811
    """A sum of squares past fp32, an infinity, a NaN, zeros without eps: NaN in the whole row, not zeros; the other
    rows as without them."""
    say(f"norm bf16 rows without a norm h={h}")
    x = inputs(9, h, False, None, 26)[0]
    alone = torch.empty((9, h), dtype=BF16, device="cuda")
    dg.rmsnorm_bf16(x, None, alone, 0.0)
    bad = x.clone()
    bad[1] = 1e30
    bad[3, h - 1] = float("inf")
    bad[4, 0] = float("nan")
    bad[6] = 0
    bad[7] = -3e38
    for total in (None, torch.empty_like(bad)):
        y = torch.full_like(bad, 7.0)
        dg.rmsnorm_bf16(bad, None, y, 0.0, None, total)
        assert y[[1, 3, 4, 6, 7]].isnan().all()
        assert torch.equal(y[[0, 2, 5, 8]], alone[[0, 2, 5, 8]])
