"""Tokens sorted by expert and back on the GPU: the rows against a walk over the
slots on the host, the copies bit for bit, sums and gradients against the
formulas in 64 bits.

Tolerances (before the first run).  combine adds at most 17 terms in fp32:
    |y - ref| <= 2^-8 |ref| + 2^-19 (|residual| + sum |w o|)      (17 roundings of 2^-24)
    dout: w dy rounded to fp32 and to bf16: (2^-8 + 2^-23) |w dy|
    |dweights - ref| <= 2^-17 sum |dy o|   (at most 8 * 32 + 6 + 8 roundings of 2^-24, sizes to 2^17 columns)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F32, F64, FP8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def by_hand(ids, e, limit, masked):
    """Rows of the slots, m_indices (contiguous) and rows per expert."""
    flat = ids.cpu().numpy().reshape(-1)
    rows = np.full(flat.shape, -1, np.int64)
    counts, start = np.zeros(e, np.int64), 0
    m_indices = None if masked else np.full(limit, -1, np.int64)
    order = np.argsort(flat, kind="stable")
    ordered = flat[order]
    for x in range(e):
        at = order[np.searchsorted(ordered, x):np.searchsorted(ordered, x, side="right")]
        if masked:
            got = x * limit + np.arange(min(len(at), limit))
        else:
            got = start + np.arange(len(at))
            got = got[got < limit]
            m_indices[got] = x
            start += (len(at) + 127) // 128 * 128
        rows[at[:len(got)]] = got
        counts[x] = len(got)
    return rows.reshape(ids.shape), m_indices, counts


def routing(t, k, e, seed=0, kind="spread"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        return torch.full((t, k), e - 1, dtype=torch.int32, device="cuda")
    if kind == "none":
        ids = torch.randint(-5, 0, (t, k), generator=g, device="cuda")
        ids[::2] = e + 3
        return ids.to(torch.int32)
    ids = torch.randint(0, e, (t, k), generator=g, device="cuda")
    if kind == "skewed":
        ids = (ids * torch.rand((t, k), generator=g, device="cuda") ** 4).long()
    if kind == "holes":
        ids = torch.where(torch.rand((t, k), generator=g, device="cuda") < 0.4, 2 * ids - e, ids)
    return ids.to(torch.int32)


SHAPES = [(1, 1, 1), (1, 8, 256), (3, 2, 5), (64, 8, 32), (129, 16, 1024), (777, 6, 24), (1025, 8, 8), (1300, 7, 513),
          (4096, 8, 256), (9000, 1, 1024), (33001, 3, 60)]


@pytest.mark.parametrize("t,k,e", SHAPES)
@pytest.mark.parametrize("kind", ["spread", "skewed", "holes", "one", "none"])
def test_sort_contiguous(dg, t, k, e, kind):
    say(f"sort contiguous {t}x{k} of {e} {kind}")
    ids = routing(t, k, e, 1, kind)
    m = dg.moe_sort_rows(t, k, e)
    m_indices, rows = torch.full((m,), 99, dtype=torch.int32, device="cuda"), torch.full((t, k), 99, dtype=torch.int32, device="cuda")
    counts = torch.full((e,), 99, dtype=torch.int32, device="cuda")
    dg.moe_sort_contiguous(ids, e, m_indices, rows, counts)
    want = by_hand(ids, e, m, False)
    for got, w, name in zip((rows, m_indices, counts), want, ("rows", "m_indices", "counts")):
        assert np.array_equal(got.cpu().numpy(), w), name


@pytest.mark.parametrize("t,k,e", [(3, 2, 5), (64, 8, 32), (1300, 7, 513), (33001, 3, 60)])
@pytest.mark.parametrize("m", [128, 384, 1024])
def test_sort_contiguous_with_too_few_rows(dg, t, k, e, m):
    """Slots past M_total have no row, and nothing is written past it."""
    say(f"sort contiguous {t}x{k} of {e} in {m} rows")
    ids = routing(t, k, e, 2, "skewed")
    buf = torch.full((m + 256,), 99, dtype=torch.int32, device="cuda")
    rows, counts = torch.empty_like(ids), torch.empty(e, dtype=torch.int32, device="cuda")
    dg.moe_sort_contiguous(ids, e, buf[:m], rows, counts)
    want = by_hand(ids, e, m, False)
    assert np.array_equal(rows.cpu().numpy(), want[0])
    assert np.array_equal(buf[:m].cpu().numpy(), want[1]) and (buf[m:] == 99).all()
    assert np.array_equal(counts.cpu().numpy(), want[2])


@pytest.mark.parametrize("t,k,e", SHAPES)
@pytest.mark.parametrize("kind,m_max", [("spread", 64), ("skewed", 16), ("holes", 1), ("one", 7), ("none", 3),
                                        ("spread", 40000)])
def test_sort_masked(dg, t, k, e, kind, m_max):
    say(f"sort masked {t}x{k} of {e} {kind} M_max={m_max}")
    ids = routing(t, k, e, 3, kind)
    rows, masked_m = torch.empty_like(ids), torch.full((e,), 99, dtype=torch.int32, device="cuda")
    dg.moe_sort_masked(ids, m_max, masked_m, rows)
    want = by_hand(ids, e, m_max, True)
    assert np.array_equal(rows.cpu().numpy(), want[0])
    assert np.array_equal(masked_m.cpu().numpy(), want[2])


def test_sort_of_many_slots(dg):
    """2^23 slots, the most there may be."""
    say("sort 2^23 slots")
    t, k, e = 1 << 20, 8, 300
    ids = routing(t, k, e, 4, "holes")
    m = dg.moe_sort_rows(t, k, e)
    m_indices, rows = torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty_like(ids)
    counts = torch.empty(e, dtype=torch.int32, device="cuda")
    dg.moe_sort_contiguous(ids, e, m_indices, rows, counts)
    want = by_hand(ids, e, m, False)
    assert np.array_equal(rows.cpu().numpy(), want[0])
    assert np.array_equal(m_indices.cpu().numpy(), want[1])
    assert np.array_equal(counts.cpu().numpy(), want[2])


def sorted_rows(dg, ids, e, masked, m_max=0):
    rows = torch.empty_like(ids)
    if masked:
        masked_m = torch.empty(e, dtype=torch.int32, device="cuda")
        dg.moe_sort_masked(ids, m_max, masked_m, rows)
        return rows, None, e * m_max
    m = dg.moe_sort_rows(*ids.shape, e)
    m_indices = torch.empty(m, dtype=torch.int32, device="cuda")
    dg.moe_sort_contiguous(ids, e, m_indices, rows)
    return rows, m_indices, m


def spread64(x, rows, m, fill):
    """x's rows [T, B] bytes at the rows of their slots, `fill` elsewhere."""
    out = torch.full((m, x.shape[1]), fill, dtype=x.dtype, device="cuda")
    r = rows.long().reshape(-1)
    src = torch.arange(rows.shape[0], device="cuda").repeat_interleave(rows.shape[1])
    ok = r >= 0
    out[r[ok]] = x[src[ok]]
    return out


def bytes_of(x):
    return x.view(torch.uint8).reshape(x.shape[0], -1)


DISPATCH = [(1, 1, 1, 128), (1, 8, 16, 7168), (5, 2, 4, 256), (64, 8, 32, 1024), (300, 6, 24, 2176), (1200, 3, 7, 640),
            (2000, 16, 40, 4224)]


@pytest.mark.parametrize("t,k,e,h", DISPATCH)
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "ue8m0"])
def test_dispatch(dg, t, k, e, h, masked, kind):
    say(f"dispatch {kind} {t}x{k} of {e} h={h} masked={masked}")
    ids = routing(t, k, e, 5, "holes")
    rows, m_indices, m = sorted_rows(dg, ids, e, masked, 48)
    g = torch.Generator(device="cuda").manual_seed(6)
    layout = (e, m // e) if masked else (m,)
    if kind == "bf16":
        x = torch.randn((t, h), generator=g, device="cuda").to(BF16)
        a = torch.full((*layout, h), 3.0, dtype=BF16, device="cuda")
        dg.moe_dispatch_bf16(x, rows, a)
        a = a.view(m, h)
        assert torch.equal(a, spread64(x, rows, m, 3.0))
        return
    x = torch.randint(0, 256, (t, h), generator=g, device="cuda", dtype=torch.uint8)
    words = h // 128 if kind == "fp8" else (h + 511) // 512
    s = torch.randint(-2 ** 31, 2 ** 31 - 1, (t, words), generator=g, device="cuda", dtype=torch.int32)
    a = torch.full((*layout, h), 3, dtype=torch.uint8, device="cuda")
    sa = torch.full((*layout, words), 3, dtype=torch.int32, device="cuda")
    as_scales = (lambda v: v) if kind == "ue8m0" else (lambda v: v.view(F32))
    dg.moe_dispatch_fp8((x.view(FP8), as_scales(s)), rows, (a.view(FP8), as_scales(sa)))
    assert torch.equal(a.view(m, h), spread64(x, rows, m, 3))
    assert torch.equal(sa.view(m, words), spread64(s, rows, m, 3))


@pytest.mark.parametrize("t,k,e,h", DISPATCH)
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_dispatch_with_padding_of_zeros(dg, t, k, e, h, kind):
    """The rows of -1 in the segments' last blocks are zeros; those behind the last segment stay."""
    say(f"dispatch padding {kind} {t}x{k} of {e} h={h}")
    ids = routing(t, k, e, 7, "holes")
    rows, m_indices, m = sorted_rows(dg, ids, e, False)
    used = (m_indices.view(-1, 128) >= 0).any(1).repeat_interleave(128)
    free = ~used
    g = torch.Generator(device="cuda").manual_seed(8)
    if kind == "bf16":
        x = torch.randn((t, h), generator=g, device="cuda").to(BF16)
        a = torch.full((m, h), float("nan"), dtype=BF16, device="cuda")
        dg.moe_dispatch_bf16(x, rows, a, m_indices)
        want = spread64(x, rows, m, 0.0)
        assert torch.equal(a[used], want[used]) and a[free].isnan().all()
        return
    x = torch.randint(0, 256, (t, h), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.rand((t, h // 128), generator=g, device="cuda")
    a, sa = torch.full((m, h), 9, dtype=torch.uint8, device="cuda"), torch.full((m, h // 128), 9.0, device="cuda")
    dg.moe_dispatch_fp8((x.view(FP8), s), rows, (a.view(FP8), sa), m_indices)
    for got, src in ((a, x), (sa, s)):
        assert torch.equal(got[used], spread64(src, rows, m, 0)[used]) and (got[free] == 9).all()


def test_rows_outside_the_layout(dg):
    """Rows at or past M, and negative ones of any size, are no rows."""
    say("rows outside the layout")
    t, k, h, m = 6, 4, 64, 128
    rows = torch.tensor([[0, 128, -1, 5], [2 ** 31 - 1, 1, -2 ** 31, 6], [-7, 129, 4000, 200], [2, 3, 127, 128],
                         [10, 11, 12, 13], [-1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    fine = torch.where((rows >= 0) & (rows < m), rows, torch.full_like(rows, -1))
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((t, h), generator=g, device="cuda").to(BF16)
    a = torch.zeros((m, h), dtype=BF16, device="cuda")
    dg.moe_dispatch_bf16(x, rows, a)
    assert torch.equal(a, spread64(x, fine, m, 0.0))
    o = torch.randn((m, h), generator=g, device="cuda").to(BF16)
    w = torch.randn((t, k), generator=g, device="cuda")
    w[rows != fine] = float("nan")  # a slot without a row adds nothing, whatever its weight
    y, want = torch.empty((t, h), dtype=BF16, device="cuda"), torch.empty((t, h), dtype=BF16, device="cuda")
    dg.moe_combine_bf16(o, rows, y, w)
    dg.moe_combine_bf16(o, fine, want, torch.nan_to_num(w))
    assert torch.equal(y, want) and (y[5] == 0).all()
    do, dw = torch.zeros_like(o), torch.empty_like(w)
    do2, dw2 = torch.zeros_like(o), torch.empty_like(w)
    dg.moe_combine_bf16_backward(x, o, rows, w, do, dw)
    dg.moe_combine_bf16_backward(x, o, fine, torch.nan_to_num(w), do2, dw2)
    assert torch.equal(do, do2) and torch.equal(dw, dw2) and (dw[rows != fine] == 0).all()


def gathered(o, rows):
    v = o[rows.clamp(min=0).long()].to(F64)
    return torch.where((rows >= 0)[:, :, None], v, torch.zeros((), dtype=F64, device="cuda"))


@pytest.mark.parametrize("t,k,e,h", [(1, 1, 1, 8), (1, 8, 16, 7168), (7, 3, 4, 520), (64, 8, 32, 1024), (777, 6, 24, 2048),
                                     (90, 16, 40, 1000), (33, 9, 12, 4104)])
@pytest.mark.parametrize("weights,residual", [(True, True), (False, True), (True, False), (False, False)])
def test_combine(dg, t, k, e, h, weights, residual):
    say(f"combine {t}x{k} of {e} h={h} weights={weights} residual={residual}")
    rows, _, m = sorted_rows(dg, routing(t, k, e, 10, "holes"), e, False)
    g = torch.Generator(device="cuda").manual_seed(11)
    o = torch.full((m, h), float("nan"), dtype=BF16, device="cuda")  # (rows that no slot takes are not read)
    o[rows[rows >= 0].long()] = torch.randn((int((rows >= 0).sum()), h), generator=g, device="cuda").to(BF16)
    w = torch.randn((t, k), generator=g, device="cuda") if weights else None
    r = torch.randn((t, h), generator=g, device="cuda").to(BF16) if residual else None
    y = torch.full((t, h), float("nan"), dtype=BF16, device="cuda")
    assert dg.moe_combine_bf16(o, rows, y, w, r) is y
    terms = gathered(o, rows) * (1 if w is None else w.to(F64)[:, :, None])
    want, size = terms.sum(1), terms.abs().sum(1)
    if r is not None:
        want, size = want + r.to(F64), size + r.to(F64).abs()
    assert ((y.to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * size).all()
    if residual:
        dg.moe_combine_bf16(o, rows, r, w, r)
        assert torch.equal(r, y)


def test_combine_strided_rows(dg):
    say("combine strided")
    t, k, e, h, ld = 31, 4, 6, 264, 280
    rows, _, m = sorted_rows(dg, routing(t, k, e, 12), e, True, 24)
    g = torch.Generator(device="cuda").manual_seed(13)
    o = torch.randn((e, 24, h), generator=g, device="cuda").to(BF16)
    res = torch.randn((t, ld), generator=g, device="cuda").to(BF16)
    out = torch.full((t, ld), 7.0, dtype=BF16, device="cuda")
    dg.moe_combine_bf16(o, rows, out[:, 8:8 + h], None, res[:, 16:])
    want = torch.empty((t, h), dtype=BF16, device="cuda")
    dg.moe_combine_bf16(o, rows, want, None, res[:, 16:].contiguous())
    assert torch.equal(out[:, 8:8 + h], want) and (out[:, :8] == 7).all() and (out[:, 8 + h:] == 7).all()
    a, b = torch.zeros((m, h), dtype=BF16, device="cuda"), torch.zeros((m, h), dtype=BF16, device="cuda")
    dg.moe_dispatch_bf16(res[:, 16:], rows, a)
    dg.moe_dispatch_bf16(res[:, 16:].contiguous(), rows, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("t,k,e,h", [(1, 1, 1, 8), (1, 8, 16, 7168), (7, 3, 4, 520), (64, 8, 32, 1024), (777, 6, 24, 2048),
                                     (90, 16, 40, 1000), (33, 9, 12, 4104), (3, 2, 2, 131072)])
@pytest.mark.parametrize("weights", [True, False])
def test_backward(dg, t, k, e, h, weights):
    say(f"combine backward {t}x{k} of {e} h={h} weights={weights}")
    rows, m_indices, m = sorted_rows(dg, routing(t, k, e, 14, "holes"), e, False)
    used = (m_indices.view(-1, 128) >= 0).any(1).repeat_interleave(128)
    g = torch.Generator(device="cuda").manual_seed(15)
    o = torch.randn((m, h), generator=g, device="cuda").to(BF16)
    dy = torch.randn((t, h), generator=g, device="cuda").to(BF16)
    w = torch.randn((t, k), generator=g, device="cuda") if weights else None
    do, dw = torch.full((m, h), float("nan"), dtype=BF16, device="cuda"), torch.full((t, k), float("nan"), device="cuda")
    dg.moe_combine_bf16_backward(dy, o, rows, w, do, dw, m_indices)
    v, d = gathered(o, rows), dy.to(F64)[:, None, :]
    assert ((dw.to(F64) - (v * d).sum(2)).abs() <= 2.0 ** -17 * (v * d).abs().sum(2)).all()
    want = torch.zeros((m, h), dtype=F64, device="cuda")
    ok = rows >= 0
    want[rows[ok].long()] = (d * (1 if w is None else w.to(F64)[:, :, None])).expand(t, k, h)[ok]
    assert ((do.to(F64) - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs())[used].all() and do[~used].isnan().all()
    # one of the two alone, without the padding, and dout over o
    one, two = torch.full_like(do, 5.0), torch.empty_like(dw)
    dg.moe_combine_bf16_backward(dy, o, rows, w, do=one)
    dg.moe_combine_bf16_backward(dy, o, rows, w, dweights=two)
    taken = m_indices >= 0
    assert torch.equal(one[taken], do[taken]) and (one[~taken] == 5).all() and torch.equal(two, dw)
    dg.moe_combine_bf16_backward(dy, o, rows, w, do=o, dweights=two)
    assert torch.equal(o[taken], do[taken]) and torch.equal(two, dw)
    # dispatch's own gradient
    da = torch.randn((m, h), generator=g, device="cuda").to(BF16)
    dx = torch.empty((t, h), dtype=BF16, device="cuda")
    dg.moe_dispatch_bf16_backward(da, rows, dx)
    v = gathered(da, rows)
    assert ((dx.to(F64) - v.sum(1)).abs() <= 2.0 ** -8 * v.sum(1).abs() + 2.0 ** -19 * v.abs().sum(1)).all()


def test_gradients_against_differences(dg):
    """y = combine(w, dispatch(x) + c): along random directions of x, w and o the gradients' inner products against
    differences in 64 bits (the function is linear in each, so a central difference is exact but for rounding)."""
    say("moe rows differences")
    t, k, e, h = 19, 3, 5, 96
    rows, m_indices, m = sorted_rows(dg, routing(t, k, e, 16, "holes"), e, False)
    g = torch.Generator(device="cuda").manual_seed(17)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, c, dy, w = rn(t, h).to(BF16), rn(m, h).to(BF16), rn(t, h).to(BF16), rn(t, k)
    a = torch.zeros((m, h), dtype=BF16, device="cuda")
    dg.moe_dispatch_bf16(x, rows, a, m_indices)
    o = (a.float() + c.float()).to(BF16)
    do, dw, dx = torch.zeros((m, h), dtype=BF16, device="cuda"), torch.empty((t, k), device="cuda"), torch.empty_like(x)
    dg.moe_combine_bf16_backward(dy, o, rows, w, do, dw, m_indices)
    dg.moe_dispatch_bf16_backward(do, rows, dx)
    # L(x, w) with o's rounding held fixed: o = dispatch(x) + (o - a)
    fixed = o.to(F64) - a.to(F64)
    ok = (rows >= 0)[:, :, None]

    def loss(xx, ww):
        oo = torch.where(ok, xx[:, None, :] + fixed[rows.clamp(min=0).long()], torch.zeros((), dtype=F64, device="cuda"))
        return (dy.to(F64)[:, None, :] * ww[:, :, None] * oo).sum()

    for _ in range(4):
        ex, ew = rn(t, h).to(F64), rn(t, k).to(F64)
        for direction, grad, slack in ((ex, dx, 2.0 ** -8 * 2 * (k * dy.to(F64).abs() * w.to(F64).abs().amax(1, keepdim=True))),
                                       (ew, dw, 2.0 ** -17 * (dy.to(F64).abs()[:, None, :] * o.to(F64).abs().amax(0)).sum(2))):
            # (dx: do rounded to bf16, k terms, then dx itself: two roundings of at most k |w dy| 2^-8 each)
            args = lambda s: (x.to(F64) + s * ex, w.to(F64)) if direction is ex else (x.to(F64), w.to(F64) + s * ew)
            diff = (loss(*args(0.5)) - loss(*args(-0.5)))
            got = (grad.to(F64) * direction).sum()
            assert abs(got - diff) <= (slack * direction.abs()).sum() + 1e-9


def test_offsets_past_32_bits(dg):
    """A layout of more than 2^32 bytes, with rows at its end."""
    say("moe rows 64-bit offsets")
    t, h, m = 5, 16384, 140032  # 4.6 GB
    g = torch.Generator(device="cuda").manual_seed(18)
    rows = torch.tensor([[m - 1, 0], [65536, 65535], [131071, 131072], [m - 2, 7], [-1, 131073]], dtype=torch.int32,
                        device="cuda")
    x = torch.randn((t, h), generator=g, device="cuda").to(BF16)
    a = torch.zeros((m, h), dtype=BF16, device="cuda")
    dg.moe_dispatch_bf16(x, rows, a)
    for i in range(t):
        for r in rows[i].tolist():
            if r >= 0:
                assert torch.equal(a[r], x[i])
    y = torch.empty_like(x)
    dg.moe_combine_bf16(a, rows, y)
    assert torch.equal(y[:4], (2 * x[:4].float()).to(BF16)) and torch.equal(y[4], x[4])
    dw = torch.empty((t, 2), device="cuda")
    dg.moe_combine_bf16_backward(x, a, rows, None, a, dw)
    assert (dw[:4, 0] == dw[:4, 1]).all() and dw[4, 0] == 0 and torch.equal(a[m - 1], x[0])


def test_more_tokens_than_workgroups(dg):
    """2^21 + 3 tokens: a workgroup of the backward pass takes several; and 2^26 + 128 rows of padding."""
    say("moe rows 2^21 + 3 tokens")
    t, h = (1 << 21) + 3, 8
    g = torch.Generator(device="cuda").manual_seed(19)
    rows = torch.randperm(t, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    dy = torch.randn((t, h), generator=g, device="cuda").to(BF16)
    o, w = torch.randn((t, h), generator=g, device="cuda").to(BF16), torch.randn((t, 1), generator=g, device="cuda")
    do, dw = torch.empty_like(o), torch.full_like(w, float("nan"))
    dg.moe_combine_bf16_backward(dy, o, rows, w, do, dw)
    at = rows[:, 0].long()
    assert torch.equal(do[at], (w * dy.float()).to(BF16))
    want = (dy.to(F64) * o[at].to(F64))
    assert ((dw[:, 0].to(F64) - want.sum(1)).abs() <= 2.0 ** -17 * want.abs().sum(1)).all()
    m = (1 << 26) + 128
    mi = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    mi[::128] = 0
    a = torch.ones((m, 8), dtype=BF16, device="cuda")
    dg.moe_dispatch_bf16(dy[:1], torch.tensor([[-1]], dtype=torch.int32, device="cuda"), a, mi)
    assert (a[::128] == 1).all() and a.float().sum() == 8 * (m // 128)


def test_same_bits_every_time_and_captured(dg):
    say("moe rows captured")
    t, k, e, h = 1500, 8, 33, 512  # (more than one chunk)
    ids = routing(t, k, e, 20, "skewed")
    g = torch.Generator(device="cuda").manual_seed(21)
    x, w = torch.randn((t, h), generator=g, device="cuda").to(BF16), torch.rand((t, k), generator=g, device="cuda")
    m = dg.moe_sort_rows(t, k, e)
    rows, m_indices = torch.empty_like(ids), torch.empty(m, dtype=torch.int32, device="cuda")
    a, do = torch.zeros((m, h), dtype=BF16, device="cuda"), torch.zeros((m, h), dtype=BF16, device="cuda")
    y, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(max(1, dg.moe_sort_workspace(t, k, e)), dtype=torch.uint8, device="cuda")

    def step():
        dg.moe_sort_contiguous(ids, e, m_indices, rows, workspace=ws)
        dg.moe_dispatch_bf16(x, rows, a, m_indices)
        dg.moe_combine_bf16(a, rows, y, w, x)
        dg.moe_combine_bf16_backward(x, a, rows, w, do, dw, m_indices)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        ids.copy_(routing(t, k, e, 30 + n, "holes"))
        for o in (a, do, y, dw, rows, m_indices):
            o.zero_()
        graph.replay()
        got = [o.clone() for o in (rows, m_indices, a, y, do, dw)]
        torch.cuda.synchronize()
        a.zero_(), do.zero_()
        step()
        assert all(torch.equal(p, q) for p, q in zip(got, (rows, m_indices, a, y, do, dw))), n


def test_two_streams_at_once(dg):
    """Two sorts with their own buffers on two streams give what each gives alone."""
    say("moe rows two streams")
    t, k, e = 4000, 8, 100
    both = []
    for n in range(2):
        ids = routing(t, k, e, 40 + n, "skewed")
        m = dg.moe_sort_rows(t, k, e)
        both.append((ids, torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty_like(ids)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(5):
        for st, (ids, mi, rows) in zip(streams, both):
            with torch.cuda.stream(st):
                dg.moe_sort_contiguous(ids, e, mi, rows)
    torch.cuda.synchronize()
    for ids, mi, rows in both:
        want = by_hand(ids, e, mi.shape[0], False)
        assert np.array_equal(rows.cpu().numpy(), want[0]) and np.array_equal(mi.cpu().numpy(), want[1])


def test_refusals_of_the_binding(dg):
    ids = routing(4, 2, 3)
    m = dg.moe_sort_rows(4, 2, 3)
    mi, rows = torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty_like(ids)
    x, a = torch.zeros((4, 256), dtype=BF16, device="cuda"), torch.zeros((m, 256), dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        dg.moe_sort_contiguous(ids.long(), 3, mi, rows)
    with pytest.raises(ValueError):
        dg.moe_sort_contiguous(ids, 3, mi, rows[:3])
    with pytest.raises(ValueError):
        dg.moe_sort_contiguous(ids, 3, mi, rows, counts=torch.empty(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(dg.DGError):
        dg.moe_sort_contiguous(ids, 3, mi[:100], rows)
    with pytest.raises(ValueError):
        dg.moe_sort_masked(ids.t(), 8, torch.empty(3, dtype=torch.int32, device="cuda"), rows)
    with pytest.raises(ValueError):
        dg.moe_dispatch_bf16(x, rows[:3], a)
    with pytest.raises(ValueError):
        dg.moe_dispatch_bf16(x, rows, a[:, :128])
    with pytest.raises(ValueError):
        dg.moe_dispatch_bf16(x, rows, a, mi[:128 if m > 128 else 64])
    with pytest.raises(TypeError):
        dg.moe_dispatch_fp8((x[:, :128].contiguous().view(torch.uint8), torch.zeros((4, 2), device="cuda")), rows,
                            (a[:, :128].contiguous().view(torch.uint8), torch.zeros((m, 2), device="cuda", dtype=torch.int32)))
    with pytest.raises(ValueError):
        dg.moe_combine_bf16(a, rows, x, torch.ones((4, 3), device="cuda"))
    with pytest.raises(ValueError):
        dg.moe_combine_bf16_backward(x, a, rows, None, a[:128 if m > 128 else 64])
