"""The linear layer (GEMM with bias, activation and residual; BF16 and FP8) and
its backward pass on the GPU against the formulas in 64 bits.

Tolerances (before the first run), with c = |A|.|B|^T + |bias| (absolute
products): fp32 sums of the matrix unit and of at most 2^7 partials stay within
2^-16 c.  The activations' slopes are below 1.2 and their own error below
2^-20 of the argument.  A rounding to bf16 (8 significant bits: half a unit in
the last place of 2^-7) costs up to 2^-8 of the value.  So
    |pre - ref| <= 2^-16 c + 2^-8 |ref|
    |C - ref|   <= 1.2 2^-16 c + 2^-20 |pre| + r |ref|,  r = 2^-8 (bf16) or 2^-22 (fp32)
Backward, with d = dpre in 64 bits from the stored pre: the slopes' error is
below 2^-18, d is rounded to bf16 (2^-8), and the products of absolute values
bound the rest:
    |da - ref| <= (2^-8 + 2^-16) |d|.|B| + 2^-18 |dc|.|B| + 2^-8 |ref|, db likewise,
    |dbias - ref| <= sum 2^-16 |d| + 2^-18 |dc|."""
from __future__ import annotations

import os

import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
TILES = ["256x256x2x4", "256x128x4x2", "128x128x2x2", "64x128x2x2", "64x64x2x2"]


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
    if a == "relu":
        return torch.relu(x)
    if a == "gelu":
        return torch.nn.functional.gelu(x)
    if a == "gelu_tanh":
        return torch.nn.functional.gelu(x, approximate="tanh")
    if a == "silu":
        return torch.nn.functional.silu(x)
    return x


def slope64(x, a):
    x = x.detach().clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act64(x, a).sum(), x)
    return g


def sentinel(m, n, dtype=BF16, ld=None):
    """[m, n] view of a wider buffer filled with a NaN pattern."""
    buf = torch.full((m, ld or n), float("nan"), dtype=dtype, device="cuda")
    return buf[:, :n], buf


def worst(got, ref, bound, what):
    got = got.to(F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    w = ((got - ref).abs() / (bound + 1e-30)).max().item()
    assert w <= 1, f"{what}: {w:.3g} times the bound"


def forward_case(dg, m, n, k, act="none", bias=None, residual=False, pre=False, out=BF16, fp8=False, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * m + n)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    if fp8:
        # random codes with |value| up to 2 and scales of another binade per group
        qa, qb = rn(m, k).clamp(-3, 3).to(torch.float8_e4m3fn), rn(n, k).clamp(-3, 3).to(torch.float8_e4m3fn)
        sa = torch.exp2(torch.randint(-3, 3, (m, k // 128), generator=g, device="cuda").float()) * 1.37
        sb = torch.exp2(torch.randint(-3, 3, ((n + 127) // 128, k // 128), generator=g, device="cuda").float()) * 0.71 / k ** 0.5
        a64 = qa.float().to(F64) * sa.to(F64).repeat_interleave(128, 1)
        b64 = qb.float().to(F64) * sb.to(F64).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    else:
        ab, bb = rn(m, k + pad).to(BF16), (rn(n, k + pad) / k ** 0.5).to(BF16)
        qa, qb = ab[:, :k], bb[:, :k]
        a64, b64 = qa.to(F64), qb.to(F64)
    bt = None if bias is None else rn(n).to(bias)
    res = rn(m, n + pad).to(BF16)[:, :n] if residual else None
    o, obuf = sentinel(m, n, out, n + pad)
    pr, pbuf = sentinel(m, n, BF16, n + pad) if pre else (None, None)
    if fp8:
        dg.gemm_fp8_nt_epilogue((qa, sa), (qb, sb), o, bt, act, res, pr)
    else:
        dg.gemm_bf16_nt_epilogue(qa, qb, o, bt, act, res, pr)
    torch.cuda.synchronize()
    z = a64 @ b64.t()
    c = a64.abs() @ b64.abs().t()
    if bt is not None:
        z, c = z + bt.to(F64), c + bt.to(F64).abs()
    ref = act64(z, act)
    if residual:
        ref = ref + res.to(F64)
    r = 2.0 ** -8 if out == BF16 else 2.0 ** -22
    what = f"{m}x{n}x{k} {act} bias={bias} res={residual} pre={pre} {out} fp8={fp8}"
    worst(o, ref, 1.2 * 2.0 ** -16 * c + 2.0 ** -20 * z.abs() + r * ref.abs(), what)
    if pre:
        worst(pr, z, 2.0 ** -16 * c + 2.0 ** -8 * z.abs(), what + " pre")
    if pad:
        assert torch.isnan(obuf[:, n:].float()).all() and (not pre or torch.isnan(pbuf[:, n:].float()).all()), \
            what + ": wrote past the row"
    return o


SIZES = [(1, 1, 8), (1, 7168, 256), (3, 17, 40), (16, 130, 1032), (17, 64, 520), (33, 100, 128), (64, 257, 2056),
         (65, 66, 72), (100, 2111, 200), (130, 256, 1032), (257, 390, 64), (300, 520, 8)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("variant", range(5))
def test_forward_bf16(dg, m, n, k, variant):
    say(f"linear {m}x{n}x{k} v{variant}")
    forward_case(dg, m, n, k, ACTS[variant], bias=[None, F32, BF16][variant % 3], residual=variant % 2 == 1,
                 pre=variant >= 2, out=F32 if variant in (0, 3) else BF16, pad=8 if variant in (1, 4) else 0)


@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 300, 1152), (16, 2112, 256), (29, 129, 384), (64, 128, 2176),
                                   (65, 130, 128), (150, 2111, 640), (300, 520, 256)])
@pytest.mark.parametrize("variant", range(5))
def test_forward_fp8(dg, m, n, k, variant):
    say(f"linear fp8 {m}x{n}x{k} v{variant}")
    forward_case(dg, m, n, k, ACTS[variant], bias=[BF16, None, F32][variant % 3], residual=variant % 2 == 0,
                 pre=variant in (1, 4), out=F32 if variant == 2 else BF16, fp8=True)


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("m,n,k,splits", [(5, 9, 64, None), (300, 390, 200, None), (257, 257, 1032, None),
                                          (40, 300, 1544, 3), (130, 129, 712, 4)])
def test_forward_tiles(dg, force, tile, m, n, k, splits):
    force(tile, splits)
    say(f"linear tile {tile} {m}x{n}x{k} splits={splits}")
    o = forward_case(dg, m, n, k, "gelu", bias=F32, residual=True, pre=True)
    again = forward_case(dg, m, n, k, "gelu", bias=F32, residual=True, pre=True)
    assert torch.equal(o, again), "not deterministic"


def test_many_tiles_per_workgroup(dg, force):
    for tile in TILES:
        force(tile)
        say(f"linear many tiles {tile}")
        forward_case(dg, 2048 + 40, 8192 + 24, 72, "silu", bias=F32)


# tiles by one or two groups of waves that share K
TILES_K = [f"{t}x{w}" for t in ("128x128x2x2", "64x128x2x2", "64x64x2x2") for w in (1, 2)]


@pytest.mark.parametrize("tile", TILES_K)
@pytest.mark.parametrize("m,n,k,splits,fits", [(5, 9, 64, None, 0), (70, 200, 72, None, 0), (300, 390, 200, None, 0),
                                               (257, 264, 1032, None, 0), (130, 129, 712, 4, 0), (65, 128, 8, None, 0),
                                               (1100, 2056, 136, None, 8)])
def test_forward_tiles_by_groups(dg, force, tile, m, n, k, splits, fits):
    force(tile, splits)
    say(f"linear tile {tile} {m}x{n}x{k} splits={splits}")
    o = forward_case(dg, m, n, k, "gelu", bias=F32, residual=True, pre=True, pad=fits)
    again = forward_case(dg, m, n, k, "gelu", bias=F32, residual=True, pre=True, pad=fits)
    assert torch.equal(o, again), "not deterministic"


@pytest.mark.parametrize("tile", TILES_K)
def test_backward_parts_by_groups(dg, force, tile):
    force(tile)
    say(f"linear backward tile {tile}")
    for which in ((True, False, True), (False, True, False)):
        for m, n, k in ((300, 260, 392), (713, 333, 264), (65, 8, 200)):
            backward_case(dg, m, n, k, "silu", which=which)


@pytest.mark.parametrize("m,n,k", [(1, 64, 128), (19, 283, 2816), (64, 4500, 256), (65, 70, 3840), (300, 256, 1024),
                                   (700, 1030, 512)])
def test_fp8_with_fp32_result_is_that_exact(dg, m, n, k):
    """An fp32 result of FP8 operands is off by fp32 rounding alone: K additions,
    each rounding a partial sum no larger than the result by 2^-24 at most, in
    independent directions -- sqrt(K) 2^-24 of the whole.  (The FP8 matrix
    instructions by themselves are 1.5e-5 off.)"""
    say(f"linear fp8 fp32 {m}x{n}x{k}")
    g = torch.Generator(device="cuda").manual_seed(8)
    a = (100 * torch.randn((m, k), generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    b = (100 * torch.randn((n, k), generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    sa, sb = torch.ones((m, k // 128), device="cuda"), torch.ones(((n + 127) // 128, k // 128), device="cuda")
    o = torch.empty((m, n), device="cuda")
    dg.gemm_fp8_nt_epilogue((a, sa), (b, sb), o)
    ref = a.float().to(F64) @ b.float().to(F64).t()
    off = ((o.to(F64) - ref).norm() / ref.norm()).item()
    assert off <= k ** 0.5 * 2.0 ** -24, off


@pytest.mark.parametrize("m", [4, 200])
def test_residual_in_place_and_plain(dg, m):
    say(f"linear in place m={m}")
    g = torch.Generator(device="cuda").manual_seed(4)
    a = torch.randn((m, 256), generator=g, device="cuda").to(BF16)
    b = (torch.randn((96, 256), generator=g, device="cuda") / 16).to(BF16)
    r = torch.randn((m, 96), generator=g, device="cuda").to(BF16)
    o = torch.empty_like(r)
    dg.gemm_bf16_nt_epilogue(a, b, o, residual=r)
    x = r.clone()
    dg.gemm_bf16_nt_epilogue(a, b, x, residual=x)
    assert torch.equal(x, o)


@pytest.mark.parametrize("m", [3, 90])
@pytest.mark.parametrize("fp8", [False, True])
def test_nan_and_infinity_keep_their_place(dg, m, fp8):
    """A NaN in one row of A stays in that row, one in a row of B in that column."""
    say(f"linear nan m={m} fp8={fp8}")
    n, k = 70, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    a, b = torch.randn((m, k), generator=g, device="cuda"), torch.randn((n, k), generator=g, device="cuda")
    a[1, 100] = float("nan")
    b[33, 5] = float("nan")
    o = torch.empty((m, n), dtype=BF16, device="cuda")
    if fp8:
        ones = lambda r: torch.ones((r, 2), device="cuda")
        dg.gemm_fp8_nt_epilogue((a.to(torch.float8_e4m3fn), ones(m)), (b.to(torch.float8_e4m3fn), ones(1)), o,
                                activation="relu")
    else:
        dg.gemm_bf16_nt_epilogue(a.to(BF16), b.to(BF16), o, activation="relu")
    bad = torch.isnan(o.float())
    want = torch.zeros_like(bad)
    want[1, :] = True
    want[:, 33] = True
    assert torch.equal(bad, want)


def backward_case(dg, m, n, k, act, pad=0, which=(True, True, True), seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + m + 3 * n)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    a, b = rn(m, k + pad).to(BF16)[:, :k], (rn(n, k + pad) / k ** 0.5).to(BF16)[:, :k]
    dc = rn(m, n + pad).to(BF16)[:, :n]
    pre = (2 * rn(m, n + pad)).to(BF16)[:, :n] if act != "none" else None
    da, abuf = sentinel(m, k, BF16, k + pad) if which[0] else (None, None)
    db, bbuf = sentinel(n, k, BF16, k + pad) if which[1] else (None, None)
    dbias = torch.full((n,), float("nan"), device="cuda") if which[2] else None
    dg.gemm_bf16_nt_epilogue_backward(dc, a, b, pre, act, da, db, dbias)
    torch.cuda.synchronize()
    a64, b64, dc64 = a.to(F64), b.to(F64), dc.to(F64)
    d = dc64 * slope64(pre.to(F64), act) if act != "none" else dc64
    what = f"backward {m}x{n}x{k} {act} pad={pad}"
    q = 2.0 ** -8 + 2.0 ** -16
    if which[0]:
        ref = d @ b64
        worst(da, ref, q * (d.abs() @ b64.abs()) + 2.0 ** -18 * (dc64.abs() @ b64.abs()) + 2.0 ** -8 * ref.abs(), what + " da")
    if which[1]:
        ref = d.t() @ a64
        worst(db, ref, q * (d.t().abs() @ a64.abs()) + 2.0 ** -18 * (dc64.t().abs() @ a64.abs()) + 2.0 ** -8 * ref.abs(),
              what + " db")
    if which[2]:
        worst(dbias, d.sum(0), 2.0 ** -16 * d.abs().sum(0) + 2.0 ** -18 * dc64.abs().sum(0), what + " dbias")
    if pad:
        for buf, w in ((abuf, k), (bbuf, k)):
            assert buf is None or torch.isnan(buf[:, w:].float()).all(), what + ": wrote past the row"
    return da, db, dbias


@pytest.mark.parametrize("m,n,k", [(1, 1, 8), (5, 64, 16), (63, 17, 40), (64, 130, 256), (129, 1161, 72),
                                   (257, 100, 520), (200, 333, 1032), (517, 65, 136)])
@pytest.mark.parametrize("act", ACTS)
def test_backward(dg, m, n, k, act):
    say(f"linear backward {m}x{n}x{k} {act}")
    got = backward_case(dg, m, n, k, act, pad=8 if (m + n) % 2 else 0)
    again = backward_case(dg, m, n, k, act, pad=8 if (m + n) % 2 else 0)
    assert all(torch.equal(x, y) for x, y in zip(got, again)), "not deterministic"


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("splits", [None, 3])
def test_backward_tiles(dg, force, tile, splits):
    force(tile, splits)
    say(f"linear backward tile {tile} splits={splits}")
    for m, n, k in ((300, 260, 392), (713, 333, 264)):
        backward_case(dg, m, n, k, "silu")


@pytest.mark.parametrize("which", [(True, False, False), (False, True, False), (False, False, True)])
def test_backward_parts(dg, which):
    say(f"linear backward parts {which}")
    for act in ("none", "gelu"):
        backward_case(dg, 100, 72, 64, act, which=which)


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(dg, act):
    """The stored pre-activation and the gradients against central differences
    of the layer in 64 bits, along random directions of a, b and bias.  The
    slope is taken at the rounded pre: 2^-9 |pre| |act''| off, act'' <= 1.2;
    relu's kink lies inside the step for none of these values, by choice of
    the step."""
    say(f"linear differences {act}")
    m, n, k = 48, 40, 64
    g = torch.Generator(device="cuda").manual_seed(12)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    a, b, bias, dc = rn(m, k).to(BF16), (rn(n, k) / 8).to(BF16), rn(n), rn(m, n).to(BF16)
    out, pre = torch.empty((m, n), dtype=BF16, device="cuda"), torch.empty((m, n), dtype=BF16, device="cuda")
    dg.gemm_bf16_nt_epilogue(a, b, out, bias, act, None, pre)
    da, db, dbias = torch.empty_like(a), torch.empty_like(b), torch.empty_like(bias)
    dg.gemm_bf16_nt_epilogue_backward(dc, a, b, pre, act, da, db, dbias)
    x64 = [a.to(F64), b.to(F64), bias.to(F64)]
    dc64 = dc.to(F64)

    def loss(a_, b_, c_):
        return (act64(a_ @ b_.t() + c_, act) * dc64).sum().item()

    z = x64[0] @ x64[1].t() + x64[2]
    soft = 2.0 ** -8 * z.abs() * dc64.abs() * (0 if act in ("none", "relu") else 1.2)  # bound on |d - d(rounded pre)|
    slack = [soft @ x64[1].abs(), soft.t() @ x64[0].abs(), soft.sum(0)]
    h = 2.0 ** -16
    for i, grad in enumerate((da, db, dbias)):
        v = torch.randn(x64[i].shape, generator=g, device="cuda", dtype=F64)
        if act == "relu":
            step = [torch.zeros_like(t) for t in x64]
            step[i] = v
            dz = (step[0] @ x64[1].t() if i == 0 else x64[0] @ step[1].t() if i == 1 else step[2].expand(m, n))
            assert (z.abs() > h * dz.abs()).all()  # no kink inside the step
        up, down = list(x64), list(x64)
        up[i], down[i] = x64[i] + h * v, x64[i] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = (grad.to(F64) * v).sum().item()
        # central differences: h^2 / 6 of a third derivative along v, far below the gradients' own bound
        absd = dc64.abs() * 1.2
        own = [(absd @ x64[1].abs()), (absd.t() @ x64[0].abs()), absd.sum(0)][i] * 2.0 ** -8 + 2.0 ** -8 * grad.to(F64).abs()
        bound = ((own + slack[i]) * v.abs()).sum().item() + 1e-6
        assert abs(got - diff) <= bound, (act, i, got, diff, bound)


def test_graph_and_side_stream(dg):
    """Captured calls replay with new data (K is not split under capture); a
    call on a side stream works on that stream."""
    say("linear graph")
    m, n, k = 96, 200, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = torch.randn((m, k), generator=g, device="cuda").to(BF16), torch.randn((n, k), generator=g, device="cuda").to(BF16)
    out, pre = torch.empty((m, n), dtype=BF16, device="cuda"), torch.empty((m, n), dtype=BF16, device="cuda")
    dout = torch.randn((m, n), generator=g, device="cuda").to(BF16)
    da, db, dbias = torch.empty_like(a), torch.empty_like(b), torch.empty(n, device="cuda")
    ws = torch.empty(dg.gemm_bf16_nt_epilogue_backward_workspace(m, n), dtype=torch.uint8, device="cuda")

    def step():
        dg.gemm_bf16_nt_epilogue(a, b, out, None, "gelu", None, pre)
        dg.gemm_bf16_nt_epilogue_backward(dout, a, b, pre, "gelu", da, db, dbias, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        a.copy_(torch.randn((m, k), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, pre, da, db, dbias)]
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (out, pre, da, db, dbias)):
            # eager calls may split K: another order of the same fp32 sums
            assert (x.double() - y.double()).norm() <= 2.0 ** -7 * y.double().norm()
    side = torch.cuda.Stream()
    want = out.clone()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(out, want)


def test_refusals(dg):
    z = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device="cuda")
    a, b, o = z(4, 64), z(8, 64), z(4, 8)
    f = dg.gemm_bf16_nt_epilogue
    for exc, args, kw in [
            (TypeError, (a.float(), b, o), {}), (ValueError, (a, z(8, 72), o), {}), (ValueError, (a, b, z(4, 9)), {}),
            (TypeError, (a, b, o.half()), {}), (ValueError, (a, b, o), dict(activation="tanh")),
            (TypeError, (a, b, o), dict(bias=z(8, dt=torch.float64))), (ValueError, (a, b, o), dict(bias=z(9, dt=F32))),
            (ValueError, (a, b, o), dict(residual=z(4, 9))), (TypeError, (a, b, o), dict(residual=z(4, 8, dt=F32))),
            (ValueError, (a, b, o), dict(pre=z(3, 8))), (ValueError, (z(64, 4).t(), b, o), {}),
            (ValueError, (a.cpu(), b, o), {}), (ValueError, (a, b.cpu(), o), {}), (ValueError, (a, b, o.cpu()), {}),
            (dg.DGError, (z(4, 60), z(8, 60), o), {}),            # K % 8
            (dg.DGError, (z(4, 72)[:, 4:68], b, o), {}),          # a not 16-byte aligned
            (dg.DGError, (z(4, 68)[:, :64], b, o), {}),           # rows not 16-byte apart
    ]:
        with pytest.raises(exc):
            f(*args, **kw)
    g = dg.gemm_bf16_nt_epilogue_backward
    for exc, args, kw in [
            (ValueError, (o, a, b, None, "gelu"), dict(da=z(4, 64))), (ValueError, (o, a, b), dict(da=z(4, 72))),
            (ValueError, (o, a, b), dict(db=z(4, 64))), (TypeError, (o, a, b), dict(dbias=z(8))),
            (ValueError, (o, a, b), dict(dbias=z(9, dt=F32))),
            (ValueError, (o, a, b), dict(da=z(4, 64), workspace=z(4))), (ValueError, (z(4, 9), a, b), dict(da=z(4, 64)))]:
        with pytest.raises(exc):
            g(*args, **kw)
    q, s = z(4, 128, dt=torch.uint8), torch.ones((4, 1), device="cuda")
    w, t = z(8, 128, dt=torch.uint8), torch.ones((1, 1), device="cuda")
    h = dg.gemm_fp8_nt_epilogue
    for exc, args in [(TypeError, ((a, s), (w, t), o)), (ValueError, ((q, s[:3]), (w, t), o)),
                      (ValueError, ((q, s), (w, t), z(4, 9)))]:
        with pytest.raises(exc):
            h(*args)
