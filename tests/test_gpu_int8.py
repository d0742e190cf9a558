"""The INT8 linear layer on the GPU against the formula in 64 bits.

The sums are exact, in int32 and in the reference (fp64: below 2^53).  With
p = sa sb sum, three roundings of 2^-24 (the sum to fp32 and two products), the
bias' addition, and as for the BF16 layer slopes below 1.2, activations within
2^-20 of their argument and one rounding r of the result (2^-8 or 2^-24):
    |pre - ref| <= 2^-22 |p| + 2^-23 |ref| + 2^-8 |ref|
    |C - ref|   <= 1.2 (2^-22 |p| + 2^-23 |pre|) + 2^-20 |pre| + 2^-23 |ref| + r |ref|.
The quantiser: s = amax / 127 within 2^-24, |q s - x| <= s / 2 + 2^-22 |x|."""
from __future__ import annotations

import os

import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
TILES = ["256x256x2x4", "256x128x4x2", "128x128x2x2x1", "64x128x2x2x1", "64x64x2x2x1", "128x128x2x2x2", "64x128x2x2x2",
         "64x64x2x2x2"]


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


@pytest.fixture
def force():
    def _set(tile=None, splits=None):
        for k, v in (("DG_FORCE_TILE", tile), ("DG_FORCE_SPLITS", splits)):
            os.environ.pop(k, None)
            if v is not None:
                os.environ[k] = str(v)
    yield _set
    _set()


def act64(x, a):
    return {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
            "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[a](x)


def operands(m, n, k, seed=0, stride=0, full=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(rows):
        lo = -128 if full else -127
        v = torch.randint(lo, 128, (rows, k + stride), generator=g, device="cuda", dtype=torch.int8)
        return v[:, :k]

    a, b = codes(m), codes(n)
    sa = torch.rand(m, generator=g, device="cuda") * 0.02 + 1e-3
    sb = torch.rand(n, generator=g, device="cuda") * 0.02 / k ** 0.5 + 1e-5
    return (a, sa), (b, sb)


def check(dg, m, n, k, act="none", bias=None, residual=False, pre=False, out=BF16, seed=0, stride=0, ldc=0):
    (a, sa), (b, sb) = operands(m, n, k, seed, stride)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    bv = None if bias is None else torch.randn(n, generator=g, device="cuda").to(bias)
    buf = torch.full((m, n + ldc), 7.0, dtype=out, device="cuda")
    c = buf[:, :n]
    r = torch.randn((m, n + ldc), generator=g, device="cuda").to(BF16)[:, :n] if residual else None
    p = torch.full((m, n + ldc), float("nan"), dtype=BF16, device="cuda")[:, :n] if pre else None
    assert dg.gemm_int8_nt_epilogue((a, sa), (b, sb), c, bv, act, r, p) is c
    prod = (a.to(F64) @ b.to(F64).t()) * sa.to(F64)[:, None] * sb.to(F64)
    want_pre = prod if bv is None else prod + bv.to(F64)
    off = 2.0 ** -22 * prod.abs() + 2.0 ** -23 * want_pre.abs()
    if pre:
        assert ((p.to(F64) - want_pre).abs() <= off + 2.0 ** -8 * want_pre.abs()).all(), "pre"
    want = act64(want_pre, act)
    if r is not None:
        want = want + r.to(F64)
    r1 = 2.0 ** -8 if out == BF16 else 2.0 ** -24
    bound = 1.2 * off + 2.0 ** -20 * want_pre.abs() * (act != "none") + 2.0 ** -23 * want.abs() + r1 * want.abs()
    bad = ~((c.to(F64) - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"
    assert (buf[:, n:] == 7).all()
    return c


SHAPES = [(1, 1, 16), (1, 64, 7168), (3, 100, 256), (16, 4096, 512), (17, 130, 272), (33, 257, 1040), (64, 513, 3200),
          (65, 64, 128), (100, 1000, 144), (130, 2111, 1536), (300, 129, 64), (513, 520, 2064), (1000, 768, 4096)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act,bias,residual,pre,out", [("none", None, False, False, BF16), ("silu", F32, True, True, BF16),
                                                       ("gelu", BF16, True, False, F32)])
def test_shapes(dg, m, n, k, act, bias, residual, pre, out):
    say(f"int8 {m}x{n}x{k} {act} {out}")
    check(dg, m, n, k, act, bias, residual, pre, out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [5, 200])
def test_activations(dg, m, act):
    say(f"int8 activation {act} m={m}")
    check(dg, m, 264, 512, act, F32, True, True, BF16, seed=3)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("m,n,k,ldc", [(300, 520, 1552, 0), (270, 515, 1040, 0), (129, 264, 2048, 5)])
def test_every_tile(dg, force, tile, splits, m, n, k, ldc):
    """(rows of C on 16-byte boundaries and not, edges inside a tile and inside a block of K)"""
    say(f"int8 tile {tile} splits {splits} {m}x{n}x{k}")
    force(tile, splits)
    check(dg, m, n, k, "gelu_tanh", F32, True, True, BF16, 4, ldc=ldc)
    check(dg, m, n, k, "none", None, False, False, F32, 5, ldc=ldc)


@pytest.mark.parametrize("m", [1, 7, 16, 20, 40, 64, 90])
@pytest.mark.parametrize("n,k,stride", [(72, 1664, 32), (5000, 304, 16), (33, 16, 0), (700, 8192, 48)])
def test_strided_operands(dg, m, n, k, stride):
    say(f"int8 strided {m}x{n}x{k}+{stride}")
    check(dg, m, n, k, "relu", BF16, True, False, BF16, 6, stride, 3)


@pytest.mark.parametrize("m", [4, 150])
def test_sums_reach_the_ends_of_int32(dg, m):
    """All codes -128, and -128 against 127, over the longest K."""
    say(f"int8 longest K m={m}")
    k, n = (1 << 17) - 16, 40
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    b = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    b[1::2] = 127
    sa, sb = torch.full((m,), 2.0 ** -10, device="cuda"), torch.full((n,), 2.0 ** -8, device="cuda")
    c = torch.empty((m, n), device="cuda")
    dg.gemm_int8_nt_epilogue((a, sa), (b, sb), c)
    want = torch.tensor([128 * 128 * k, -128 * 127 * k], dtype=F64, device="cuda").repeat(n // 2) * 2.0 ** -18
    assert ((c.to(F64) - want).abs() <= 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("tile,splits", [(None, None), ("64x64x2x2x1", 4), ("128x128x2x2x2", 2)])
def test_small_sums_are_exact(dg, force, tile, splits):
    """Partial sums are whole numbers of either sign, small and large: scales of one give them back, every one."""
    say(f"int8 exact sums {tile} {splits}")
    force(tile, splits)
    g = torch.Generator(device="cuda").manual_seed(7)
    for m, n, k in ((150, 91, 2048), (257, 300, 4096)):
        a = torch.randint(-2, 3, (m, k), generator=g, device="cuda", dtype=torch.int8)
        b = torch.randint(-2, 3, (n, k), generator=g, device="cuda", dtype=torch.int8)
        b[::3] *= 40
        b[5] = 0
        one = lambda x: torch.ones(x, device="cuda")
        c = torch.empty((m, n), device="cuda")
        dg.gemm_int8_nt_epilogue((a, one(m)), (b, one(n)), c)
        assert torch.equal(c.to(F64), a.to(F64) @ b.to(F64).t())


def test_special_scales(dg):
    """A NaN scale makes its row or column NaN and no other; zeros and infinities as fp32 has them."""
    say("int8 special scales")
    for m in (9, 200):
        (a, sa), (b, sb) = operands(m, 136, 256, 8)
        want = torch.empty((m, 136), device="cuda")
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), want)
        sa[3], sb[100], sb[7] = float("nan"), float("nan"), 0.0
        got = torch.empty_like(want)
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), got)
        assert got[3].isnan().all() and got[:, 100].isnan().all()
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[3], rest[:, 100], rest[:, 7] = False, False, False
        assert torch.equal(got[rest], want[rest]) and (got[[0, 1, 2, 4], 7] == 0).all()


def test_captured_gives_the_same(dg):
    """Captured calls do not split K; whole sums are the same either way."""
    say("int8 captured")
    m, n, k = 200, 264, 7168
    (a, sa), (b, sb) = operands(m, n, k, 9)
    c, eager = torch.empty((m, n), dtype=BF16, device="cuda"), torch.empty((m, n), dtype=BF16, device="cuda")
    dg.gemm_int8_nt_epilogue((a, sa), (b, sb), eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), c)
    for seed in range(3):
        a.copy_(operands(m, n, k, 20 + seed)[0][0])
        c.fill_(float("nan"))
        graph.replay()
        got = c.clone()
        torch.cuda.synchronize()
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), eager)
        assert torch.equal(got, eager)


def test_another_stream(dg):
    say("int8 another stream")
    (a, sa), (b, sb) = operands(300, 200, 4096, 10)
    want, got = (torch.empty((300, 200), dtype=BF16, device="cuda") for _ in range(2))
    dg.gemm_int8_nt_epilogue((a, sa), (b, sb), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), got)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("m,k,stride,offset", [(1, 1, 0, 0), (3, 16, 0, 0), (5, 1000, 0, 0), (7, 4100, 4, 0), (4, 1023, 0, 1),
                                               (2, 130000, 0, 0), (9, 256, 3, 2)])
def test_quantiser(dg, kind, m, k, stride, offset):
    say(f"int8 quantiser {m}x{k} {kind}")
    g = torch.Generator(device="cuda").manual_seed(11)
    buf = torch.randn(m * (k + stride) + offset, generator=g, device="cuda").to(kind)
    x = buf[offset:].view(m, k + stride)[:, :k]
    if m > 2:
        x[1] = 0
        x[2] *= 1e-30
    q, s = torch.empty((m, k), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    dg.dg_quantize_int8_rows(x, q, s)
    need = x.to(F64).abs().amax(1) / 127
    need = torch.where(need == 0, torch.ones_like(need), need)
    assert ((s.to(F64) - need).abs() <= 2.0 ** -24 * need).all()
    v = q.to(F64) * s.to(F64)[:, None]
    assert ((v - x.to(F64)).abs() <= 0.5 * s.to(F64)[:, None] + 2.0 ** -22 * x.to(F64).abs()).all()
    assert (q.to(torch.int32).abs() <= 127).all()


def test_quantiser_of_bad_rows(dg):
    say("int8 quantiser bad rows")
    for kind, k in ((BF16, 512), (F32, 513)):
        x = torch.randn((4, k), device="cuda").to(kind)
        x[1, 17], x[2, 300] = float("nan"), float("-inf")
        _, s = dg.quantize_int8_rows(x)
        assert s[1].isnan() and s[2].isnan() and not s[0].isnan() and not s[3].isnan()


def test_refusals_of_the_binding(dg):
    (a, sa), (b, sb) = operands(4, 32, 64)
    c = torch.empty((4, 32), dtype=BF16, device="cuda")
    with pytest.raises(TypeError):
        dg.gemm_int8_nt_epilogue((a.float(), sa), (b, sb), c)
    with pytest.raises(ValueError):
        dg.gemm_int8_nt_epilogue((a, sa[:3]), (b, sb), c)
    with pytest.raises(TypeError):
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb.to(BF16)), c)
    with pytest.raises(ValueError):
        dg.gemm_int8_nt_epilogue((a, sa), (b[:, :48], sb), c)
    with pytest.raises(ValueError):
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), c.t())
    with pytest.raises(ValueError):
        dg.gemm_int8_nt_epilogue((a, sa), (b, sb), c, activation="tanh")
    with pytest.raises(dg.DGError):
        dg.gemm_int8_nt_epilogue((a[:, :40], sa), (b[:, :40], sb), c)


@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("k", [8, 255, 256, 257, 500, 512, 513, 1000, 1024, 1025, 2048, 2049])
@pytest.mark.parametrize("m", [1, 17, 1023, 1025])
def test_quantiser_of_short_rows(dg, kind, k, m):
    """Rows of 16, 64 and 256 lanes, with one that is all zeros and one with a NaN."""
    say(f"int8 quantiser {m}x{k} {kind}")
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn((m, k), generator=g, device="cuda").to(kind)
    if m > 9:
        x[4] = 0
        x[9, k - 1] = float("nan")
    q, s = torch.full((m * k + 8,), 77, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    dg.dg_quantize_int8_rows(x, q[:m * k].view(m, k), s)
    assert (q[m * k:] == 77).all()
    if m > 9:
        assert s[4] == 1 and (q[4 * k:5 * k] == 0).all() and s[9].isnan()
    fine = [i for i in range(m) if i != 9]
    x, q, s = x[fine], q[:m * k].view(m, k)[fine], s[fine]
    need = x.to(F64).abs().amax(1) / 127
    need = torch.where(need == 0, torch.ones_like(need), need)
    assert ((s.to(F64) - need).abs() <= 2.0 ** -24 * need).all()
    assert ((q.to(F64) * s.to(F64)[:, None] - x.to(F64)).abs() <=
            0.5 * s.to(F64)[:, None] + 2.0 ** -22 * x.to(F64).abs()).all()


@pytest.mark.parametrize("m", [3, 600])
def test_operands_past_32_bits(dg, m):
    """Rows 4 MB apart, 2.5 GB in all, in either operand; a quantiser's rows 2 GB apart."""
    say(f"int8 rows far apart {m}")
    k, stride, n = 256, 1 << 22, 600
    (a, sa), (b, sb) = operands(m, n, k)
    far = torch.zeros((n - 1) * stride + k, dtype=torch.int8, device="cuda").as_strided((n, k), (stride, 1))
    far.copy_(b)
    c, d = torch.empty((m, n), dtype=BF16, device="cuda"), torch.empty((m, n), dtype=BF16, device="cuda")
    dg.gemm_int8_nt_epilogue((a, sa), (b, sb), c)
    dg.gemm_int8_nt_epilogue((a, sa), (far, sb), d)
    assert torch.equal(c, d)
    c, d = torch.empty((n, m), dtype=BF16, device="cuda"), torch.empty((n, m), dtype=BF16, device="cuda")
    dg.gemm_int8_nt_epilogue((b, sb), (a, sa), c)
    dg.gemm_int8_nt_epilogue((far, sb), (a, sa), d)
    assert torch.equal(c, d)
    x = torch.randn((3, 500), device="cuda").to(BF16)
    rows = torch.zeros(2 * ((1 << 30) + 8) + 500, dtype=BF16, device="cuda").as_strided((3, 500), ((1 << 30) + 8, 1))
    rows.copy_(x)
    for p, q in zip(dg.quantize_int8_rows(rows), dg.quantize_int8_rows(x)):
        assert torch.equal(p, q)
