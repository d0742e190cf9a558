"""The root-mean-square norm (bf16, FP8, INT8 outputs) and its backward pass on
the GPU against the formulas in 64 bits.

Tolerances (before the first run).  A thread sums at most 32 squares (or 32 of
them per piece), a wave and the workgroup add 6 + 8 terms, all positive, so the
sum of squares is within 2^-18 of itself (46 roundings of 2^-24, and 2^-23 for
z's own), r = its root within 2^-18 with two more, and
    |sum - z|  <= 2^-8 |z|                      (bf16; z in fp32 adds 2^-24)
    |rstd - r| <= 2^-18 r
    |y - ref|  <= 2^-17 |ref| before rounding; bf16 adds 2^-8 |ref|
    FP8: s within 2^-16 of amax/448, |q s - ref| <= 2^-4 |ref| + 2^-10 s + 2^-15 |ref|
         (half a step of e4m3; below 2^-6 its step is 2^-9)
    INT8: s within 2^-16 of amax/127, |q s - ref| <= s / 2 + 2^-15 |ref|
Backward: n = z r has 2^-24 of rounding, sums run over at most 46 terms of a row
and 64 rows or partials, so with g = w dy
    |dx - ref| <= 2^-8 |ref| + 2^-17 (r |g| + r |n| mean|g n|) + 2^-23 |dsum|
    |dw - ref| <= 2^-17 sum |dy n|."""
from __future__ import annotations

import pytest
import torch

from tests.parity import say

pytestmark = pytest.mark.gpu
BF16, F32, F64, FP8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def inputs(t, h, residual=True, weight=F32, seed=0, stride=0, offset=0):
    g = gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")

    def rows(x):
        if not stride:
            return x.to(BF16)
        buf = torch.full((t * stride + offset,), float("nan"), dtype=BF16, device="cuda")
        v = buf[offset:].view(t, stride)[:, :h]
        v.copy_(x)
        return v

    x = rows(rn(t, h) * torch.exp2(torch.randint(-3, 3, (t, 1), generator=g, device="cuda")))
    r = rows(rn(t, h) * torch.exp(rn(1, h))) if residual else None
    w = None if weight is None else (1 + 0.3 * rn(h)).to(weight)
    return x, r, w


def ref64(x, r, w, eps):
    z = x.to(F64) + (0 if r is None else r.to(F64))
    rs = 1 / torch.sqrt(z.square().mean(1) + eps)
    y = z * rs[:, None]
    return z, rs, y if w is None else y * w.to(F64)


def within(got, want, bound, what):
    bad = ~((got.to(F64) - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}"


def unpacked(s, groups):
    """Values of packed UE8M0 words [T, W], and the padding bytes."""
    b = s.view(torch.uint8).to(torch.int64)
    return torch.exp2(b[:, :groups].to(F64) - 127), b[:, groups:]


SIZES = [(1, 1), (1, 7168), (3, 8), (5, 64), (2, 127), (17, 1000), (4, 2111), (33, 512), (2, 4104), (2, 8200),
         (3, 16384), (2, 16383), (2, 5001), (700, 136), (301, 128), (77, 256), (1, 120)]


@pytest.mark.parametrize("t,h", SIZES)
@pytest.mark.parametrize("residual,weight", [(True, F32), (False, BF16), (True, None)])
def test_bf16(dg, t, h, residual, weight):
    say(f"norm bf16 {t}x{h} residual={residual} weight={weight}")
    x, r, w = inputs(t, h, residual, weight)
    out, total = (torch.full((t, h), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    rstd = torch.full((t,), float("nan"), device="cuda")
    assert dg.rmsnorm_bf16(x, w, out, 1e-5, r, total, rstd) is out
    z, rs, y = ref64(x, r, w, 1e-5)
    within(total, z, 2.0 ** -8 * z.abs() + 2.0 ** -24 * z.abs(), "sum")
    within(rstd, rs, 2.0 ** -18 * rs, "rstd")
    within(out, y, (2.0 ** -8 + 2.0 ** -16) * y.abs(), "y")


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("t,h", [(1, 128), (1, 7168), (5, 640), (37, 2048), (3, 4224), (2, 8320), (2, 16384), (301, 128), (77, 256),
                                 (9, 384)])
@pytest.mark.parametrize("residual,weight", [(True, BF16), (False, F32), (True, None)])
def test_fp8(dg, t, h, residual, weight, packed):
    say(f"norm fp8 {t}x{h} packed={packed} residual={residual} weight={weight}")
    x, r, w = inputs(t, h, residual, weight, 1)
    groups = h // 128
    q = torch.empty((t, h), dtype=FP8, device="cuda")
    s = torch.full((t, (groups + 3) // 4), -1, dtype=torch.int32, device="cuda") if packed else \
        torch.full((t, groups), float("nan"), device="cuda")
    total, rstd = torch.empty((t, h), dtype=BF16, device="cuda"), torch.empty(t, device="cuda")
    dg.rmsnorm_quantize_fp8_1x128(x, w, q, s, 1e-6, r, total, rstd)
    z, rs, y = ref64(x, r, w, 1e-6)
    within(total, z, (2.0 ** -8 + 2.0 ** -24) * z.abs(), "sum")
    within(rstd, rs, 2.0 ** -18 * rs, "rstd")
    need = y.view(t, groups, 128).abs().amax(2) / 448
    if packed:
        sv, pad = unpacked(s, groups)
        assert (pad == 0).all()
        assert (sv >= need * (1 - 2.0 ** -16)).all() and (sv < 2 * need * (1 + 2.0 ** -16)).all()
    else:
        sv = s.to(F64)
        within(sv, need, 2.0 ** -16 * need, "scales")
    se = sv.repeat_interleave(128, 1)
    within(q.float().to(F64) * se, y, (2.0 ** -4 + 2.0 ** -15) * y.abs() + 2.0 ** -10 * se, "codes")


@pytest.mark.parametrize("t,h", SIZES)
@pytest.mark.parametrize("residual,weight", [(True, BF16), (False, None)])
def test_int8(dg, t, h, residual, weight):
    say(f"norm int8 {t}x{h} residual={residual} weight={weight}")
    x, r, w = inputs(t, h, residual, weight, 2)
    q = torch.full((t, h), -128, dtype=torch.int8, device="cuda")
    s = torch.full((t,), float("nan"), device="cuda")
    total = torch.empty((t, h), dtype=BF16, device="cuda")
    dg.rmsnorm_quantize_int8(x, w, q, s, 1e-6, r, total)
    z, _, y = ref64(x, r, w, 1e-6)
    within(total, z, (2.0 ** -8 + 2.0 ** -24) * z.abs(), "sum")
    need = y.abs().amax(1) / 127
    within(s, need, 2.0 ** -16 * need, "scales")
    assert (q != -128).all() and (q.abs().amax(1) == 127).all()
    se = s.to(F64)[:, None]
    within(q.to(F64) * se, y, 0.5 * se + 2.0 ** -15 * y.abs(), "codes")


@pytest.mark.parametrize("h,stride,offset", [(256, 264, 0), (256, 264, 4), (256, 259, 0), (255, 256, 0), (1000, 1008, 8),
                                             (128, 129, 1), (5, 7, 3), (2047, 2051, 1), (8191, 8193, 5)])
def test_strided_rows_and_their_neighbours(dg, h, stride, offset):
    """Rows of longer tensors, on 16-byte boundaries or not; what lies between them stays."""
    say(f"norm strided {h} of {stride} at {offset}")
    t = 9
    x, r, w = inputs(t, h, True, F32, 3, stride, offset)
    buf = torch.full((t * stride + offset,), 7.0, dtype=BF16, device="cuda")
    total = torch.full((t * stride + offset,), 7.0, dtype=BF16, device="cuda")
    view = lambda b: b[offset:].view(t, stride)
    dg.rmsnorm_bf16(x, w, view(buf)[:, :h], 1e-6, r, view(total)[:, :h])
    z, _, y = ref64(x, r, w, 1e-6)
    within(view(buf)[:, :h], y, (2.0 ** -8 + 2.0 ** -16) * y.abs(), "y")
    within(view(total)[:, :h], z, (2.0 ** -8 + 2.0 ** -24) * z.abs(), "sum")
    for b in (buf, total):
        assert (view(b)[:, h:] == 7).all() and (b[:offset] == 7).all()
    q, s = torch.empty((t, h), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
    dg.rmsnorm_quantize_int8(x, w, q, s, 1e-6, r)
    within(q.to(F64) * s.to(F64)[:, None], y, 0.5 * s.to(F64)[:, None] + 2.0 ** -15 * y.abs(), "codes")
    if h % 128 == 0:
        q, s = torch.empty((t, h), dtype=FP8, device="cuda"), torch.empty((t, h // 128), device="cuda")
        dg.rmsnorm_quantize_fp8_1x128(x, w, q, s, 1e-6, r)
        se = s.to(F64).repeat_interleave(128, 1)
        within(q.float().to(F64) * se, y, (2.0 ** -4 + 2.0 ** -15) * y.abs() + 2.0 ** -10 * se, "fp8 codes")


@pytest.mark.parametrize("t,h", [(21, 384), (21, 2111), (768, 264), (1600, 2000)])
def test_outputs_over_inputs(dg, t, h):
    """The residual stream in place, y over x; and the backward pass over each of its inputs."""
    say(f"norm in place {t}x{h}")
    x, r, w = inputs(t, h, True, F32, 4)
    want, total = torch.empty_like(x), torch.empty_like(x)
    dg.rmsnorm_bf16(x, w, want, 1e-6, r, total)
    for which in ("residual", "x"):
        xc, rc = x.clone(), r.clone()
        sum_out, out = (rc, xc) if which == "residual" else (xc, rc)
        dg.rmsnorm_bf16(xc, w, out, 1e-6, rc, sum_out)
        assert torch.equal(sum_out, total) and torch.equal(out, want), which
    rstd = torch.rsqrt(total.float().square().mean(1) + 1e-6)
    dy, ds = inputs(t, h, True, None, 5)[:2]
    dx, dw = torch.empty_like(x), torch.empty(h, device="cuda")
    dg.rmsnorm_bf16_backward(dy, total, w, rstd, dx, dw, ds)
    for which in range(3):
        c = [dy.clone(), total.clone(), ds.clone()]
        dw2 = torch.empty_like(dw)
        dg.rmsnorm_bf16_backward(c[0], c[1], w, rstd, c[which], dw2, c[2])
        assert torch.equal(c[which], dx) and torch.equal(dw, dw2), which


def test_rows_of_zeros_and_of_bad_values(dg):
    """Rows of zeros; rows with a NaN or an infinity, or too large for their squares: NaN scales in that row
    alone; tiny rows, where eps rules; eps 0."""
    say("norm special rows")
    h = 512
    x = inputs(7, h, False, None, 6)[0]
    x[1] = 0
    x[2, 77] = float("nan")
    x[3, 500] = float("inf")
    x[4] = 1e30
    x[5] = 1e-30
    fine = [0, 1, 5, 6]
    y = ref64(x, None, None, 1e-6)[2][fine]
    out, rstd = torch.empty_like(x), torch.empty(7, device="cuda")
    dg.rmsnorm_bf16(x, None, out, 1e-6, rstd=rstd)
    within(out[fine], y, (2.0 ** -8 + 2.0 ** -16) * y.abs(), "y")
    assert out[2].isnan().all() and out[3, 500].isnan() and rstd[2].isnan() and rstd[4] == 0
    q, s = torch.empty((7, h), dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda")
    dg.rmsnorm_quantize_int8(x, None, q, s)
    assert s[[2, 3, 4]].isnan().all() and not s[fine].isnan().any() and s[1] == 1 and (q[1] == 0).all()
    se = s[fine].to(F64)[:, None]
    within(q[fine].to(F64) * se, y, 0.5 * se + 2.0 ** -15 * y.abs(), "int8")
    f, fs = torch.empty((7, h), dtype=FP8, device="cuda"), torch.empty((7, h // 128), device="cuda")
    dg.rmsnorm_quantize_fp8_1x128(x, None, f, fs)
    assert fs[[2, 3, 4]].isnan().all() and not fs[fine].isnan().any() and (fs[1] == 1).all()
    p = torch.empty((7, 1), dtype=torch.int32, device="cuda")
    dg.rmsnorm_quantize_fp8_1x128(x, None, f, p)
    b = p.view(torch.uint8)
    assert (b[[2, 3, 4]] == 255).all() and (b[fine] != 255).all() and (b[1] == 127).all()
    x = inputs(3, h, False, None, 7)[0]
    dg.rmsnorm_bf16(x, None, out[:3], 0.0)
    y = ref64(x, None, None, 0.0)[2]
    within(out[:3], y, (2.0 ** -8 + 2.0 ** -16) * y.abs(), "eps 0")


# Weights that take z w, or y itself, to the ends of fp32's range.  Besides the bounds above: a product or a scale
# below 2^-126 is rounded to a multiple of 2^-149 (half of that off), and such a scale is one unit larger.
@pytest.mark.parametrize("x_scale,w_scale", [(1.0, 2.0 ** -120), (1.0, 2.0 ** -130), (1.0, 2.0 ** -138), (2.0 ** -50, 2.0 ** -100),
                                             (2.0 ** -55, 2.0 ** -96), (2.0 ** 50, 2.0 ** 85), (1.0, 2.0 ** 110)])
@pytest.mark.parametrize("t,h", [(5, 384), (9, 128), (3, 4224), (2, 9088)])
def test_weights_at_the_ends_of_the_range(dg, t, h, x_scale, w_scale):
    say(f"norm {t}x{h} x {x_scale} w {w_scale}")
    x, _, w = inputs(t, h, False, F32, 9)
    x, w = (x.to(F32) * x_scale).to(BF16), w * w_scale
    w[::7] *= 2.0 ** -9
    y = ref64(x, None, w, 0.0)[2]
    unit = 2.0 ** -149
    q, s = torch.empty((t, h), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
    dg.rmsnorm_quantize_int8(x, w, q, s, 0.0)
    want = y.abs().amax(1) / 127
    within(s, want, 2.0 ** -16 * want + 2 * unit, "int8 scales")
    se = s.to(F64)[:, None]
    within(q.to(F64) * se, y, 0.5 * se + 2.0 ** -15 * y.abs() + unit, "int8")
    f, fs = torch.empty((t, h), dtype=FP8, device="cuda"), torch.empty((t, h // 128), device="cuda")
    dg.rmsnorm_quantize_fp8_1x128(x, w, f, fs, 0.0)
    want = y.view(t, h // 128, 128).abs().amax(2) / 448
    within(fs, want, 2.0 ** -16 * want + 2 * unit, "fp8 scales")
    se = fs.to(F64).repeat_interleave(128, 1)
    within(f.to(F64) * se, y, 2.0 ** -4 * y.abs() + 2.0 ** -10 * se + 2.0 ** -15 * y.abs() + unit, "fp8")


def test_rows_of_zeros_without_eps(dg):
    """0 / 0: NaN in every output, as in the formula."""
    say("norm of zeros, eps 0")
    x = torch.zeros((3, 256), dtype=BF16, device="cuda")
    x[1] = 1
    out, q, s = torch.empty_like(x), torch.empty((3, 256), dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    dg.rmsnorm_bf16(x, None, out, 0.0)
    dg.rmsnorm_quantize_int8(x, None, q, s, 0.0)
    f, fs, p = torch.empty((3, 256), dtype=FP8, device="cuda"), torch.empty((3, 2), device="cuda"), \
        torch.empty((3, 1), dtype=torch.int32, device="cuda")
    dg.rmsnorm_quantize_fp8_1x128(x, None, f, fs, 0.0)
    dg.rmsnorm_quantize_fp8_1x128(x, None, f, p, 0.0)
    b = p.view(torch.uint8)[:, :2]
    assert out[[0, 2]].isnan().all() and s[[0, 2]].isnan().all() and fs[[0, 2]].isnan().all() and (b[[0, 2]] == 255).all()
    assert (out[1] == 1).all() and s[1].isfinite() and fs[1].isfinite().all() and (b[1] != 255).all()


def test_more_rows_than_workgroups(dg):
    """2^21 + 3 rows: workgroups take several."""
    say("norm 2^21 + 3 rows")
    t, h = (1 << 21) + 3, 8
    x = inputs(t, h, False, None, 8)[0]
    out = torch.zeros_like(x)
    dg.rmsnorm_bf16(x, None, out)
    y = ref64(x, None, None, 1e-6)[2]
    within(out, y, (2.0 ** -8 + 2.0 ** -16) * y.abs(), "y")


def backward64(dy, z, w, r, ds):
    dy, z, r = dy.to(F64), z.to(F64), r.to(F64)[:, None]
    g = dy if w is None else dy * w.to(F64)
    n = z * r
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    slack = 2.0 ** -17 * (r * g.abs() + r * n.abs() * (g * n).abs().mean(1, keepdim=True))
    if ds is not None:
        dx = dx + ds.to(F64)
        slack = slack + 2.0 ** -23 * ds.to(F64).abs()
    return dx, slack + 2.0 ** -8 * dx.abs(), (dy * n).sum(0), 2.0 ** -17 * (dy * n).abs().sum(0)


@pytest.mark.parametrize("t,h", SIZES + [(513, 264), (1500, 65), (600, 4096), (768, 72), (769, 72), (700, 12000),
                                             (5000, 256), (777, 33), (130, 999), (5001, 128), (3000, 40),
                                             (3001, 512), (2000, 1024), (9000, 600)])
@pytest.mark.parametrize("ds,weight", [(True, F32), (False, BF16), (True, None)])
def test_backward(dg, t, h, ds, weight):
    say(f"norm backward {t}x{h} dsum={ds} weight={weight}")
    dy, d, w = inputs(t, h, ds, weight, 9)
    z = inputs(t, h, False, None, 10)[0]
    rstd = torch.rsqrt(z.float().square().mean(1) + 1e-6)
    dx, dw = torch.full((t, h), float("nan"), dtype=BF16, device="cuda"), torch.full((h,), float("nan"), device="cuda")
    dg.rmsnorm_bf16_backward(dy, z, w, rstd, dx, dw, d)
    wx, bx, ww, bw = backward64(dy, z, w, rstd, d)
    within(dx, wx, bx, "dx")
    within(dw, ww, bw, "dw")
    one, two = torch.empty_like(dx), torch.empty_like(dw)
    dg.rmsnorm_bf16_backward(dy, z, w, rstd, dx=one, dsum=d)
    dg.rmsnorm_bf16_backward(dy, z, w, rstd, dweight=two)
    assert torch.equal(one, dx) and torch.equal(two, dw)


@pytest.mark.parametrize("stride,offset", [(264, 8), (261, 3)])
def test_backward_of_strided_rows(dg, stride, offset):
    say(f"norm backward strided {stride} at {offset}")
    t, h = 14, 256
    dy, ds, w = inputs(t, h, True, BF16, 11, stride, offset)
    z = inputs(t, h, False, None, 12, stride, offset)[0]
    rstd = torch.rsqrt(z.float().square().mean(1) + 1e-6)
    buf = torch.full((t * stride + offset,), 7.0, dtype=BF16, device="cuda")
    v, dw = buf[offset:].view(t, stride), torch.empty(h, device="cuda")
    dg.rmsnorm_bf16_backward(dy, z, w, rstd, v[:, :h], dw, ds)
    wx, bx, ww, bw = backward64(dy, z, w, rstd, ds)
    within(v[:, :h], wx, bx, "dx")
    within(dw, ww, bw, "dw")
    assert (v[:, h:] == 7).all() and (buf[:offset] == 7).all()


def test_backward_against_differences(dg):
    """Along random directions: the gradients' inner product with the direction against the central difference of
    L = sum(dy y) in 64 bits (its own error: h^2 times the third derivative, 1e-8 here)."""
    say("norm backward differences")
    t, h, eps = 6, 192, 1e-5
    dy, _, w = inputs(t, h, False, F32, 13)
    z = inputs(t, h, False, None, 14)[0]
    rs = ref64(z, None, w, eps)[1]
    dx, dw = torch.empty((t, h), dtype=BF16, device="cuda"), torch.empty(h, device="cuda")
    dg.rmsnorm_bf16_backward(dy, z, w, rs.float(), dx, dw)
    bx, bw = backward64(dy, z, w, rs, None)[1::2]
    g = gen(15)
    loss = lambda zz, ww: (dy.to(F64) * zz / torch.sqrt(zz.square().mean(1, keepdim=True) + eps) * ww).sum()
    for _ in range(4):
        ez = torch.randn((t, h), generator=g, device="cuda", dtype=F64)
        ew = torch.randn((h,), generator=g, device="cuda", dtype=F64)
        d = 1e-5
        diff = (loss(z.to(F64) + d * ez, w.to(F64) + d * ew) - loss(z.to(F64) - d * ez, w.to(F64) - d * ew)) / (2 * d)
        got = (dx.to(F64) * ez).sum() + (dw.to(F64) * ew).sum()
        # (rs rounded to fp32: 2^-24 of the gradients' size, within bx and bw)
        assert abs(got - diff) <= (bx * ez.abs()).sum() + (bw * ew.abs()).sum() + 1e-5


@pytest.mark.parametrize("t,h", [(40, 512), (40, 777), (1100, 512)])
def test_captured_and_replayed(dg, t, h):
    say(f"norm captured {t}x{h}")
    x, r, w = inputs(t, h, True, F32, 16)
    dy, ds, _ = inputs(t, h, True, None, 17)
    q, s = torch.empty((t, h), dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
    total, y, dx = (torch.empty((t, h), dtype=BF16, device="cuda") for _ in range(3))
    rstd, dw = torch.empty(t, device="cuda"), torch.empty(h, device="cuda")
    ws = torch.empty(max(1, dg.rmsnorm_bf16_backward_workspace(t, h)), dtype=torch.uint8, device="cuda")

    def step():
        dg.rmsnorm_quantize_int8(x, w, q, s, 1e-6, r, total)
        dg.rmsnorm_bf16(x, w, y, 1e-6, r, total, rstd)
        dg.rmsnorm_bf16_backward(dy, total, w, rstd, dx, dw, ds, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (q, s, total, y, rstd, dx, dw)
    for k in range(3):
        nx, nr, _ = inputs(t, h, True, None, 20 + k)
        x.copy_(nx)
        r.copy_(nr)
        for o in outs:
            o.fill_(0)
        graph.replay()
        got = [o.clone() for o in outs]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), k


def test_refusals_of_the_binding(dg):
    x, r, w = inputs(4, 256, True, F32)
    out, s = torch.empty_like(x), torch.empty(4, device="cuda")
    q = torch.empty((4, 256), dtype=torch.int8, device="cuda")
    with pytest.raises(TypeError):
        dg.rmsnorm_bf16(x.float(), w, out)
    with pytest.raises(TypeError):
        dg.rmsnorm_bf16(x, w.half(), out)
    with pytest.raises(ValueError):
        dg.rmsnorm_bf16(x, w[:255], out)
    with pytest.raises(ValueError):
        dg.rmsnorm_bf16(x, w, out[:3])
    with pytest.raises(ValueError):
        dg.rmsnorm_bf16(x, w, out, residual=r[:, :128])
    with pytest.raises(ValueError):
        dg.rmsnorm_bf16(x.t(), None, out.t())
    with pytest.raises(ValueError):
        dg.rmsnorm_quantize_int8(x, w, q, s[:3])
    with pytest.raises(TypeError):
        dg.rmsnorm_quantize_int8(x, w, q.view(torch.uint8), s)
    with pytest.raises(ValueError):
        many = torch.empty((5000, 256), dtype=BF16, device="cuda")
        dg.rmsnorm_bf16_backward(many, many, w, torch.ones(5000, device="cuda"), None, torch.empty(256, device="cuda"),
                                 workspace=torch.empty(16, device="cuda"))
    with pytest.raises(dg.DGError):
        dg.rmsnorm_bf16(x, w, out, -1.0)
    with pytest.raises(dg.DGError):
        dg.rmsnorm_quantize_fp8_1x128(x[:, :192], None, q[:, :192].contiguous().view(torch.uint8),
                                      torch.empty((4, 1), device="cuda"))


def test_another_gpu_than_the_current_one(dg, monkeypatch):
    """The default stream is the current GPU's: tensors of another one are refused."""
    x, out = inputs(4, 256, False, None)[0], torch.empty((4, 256), dtype=BF16, device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    q, s = torch.zeros((4, 256), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    monkeypatch.setattr(dg, "_current_device", lambda: 1)
    for call in (lambda: dg.rmsnorm_bf16(x, None, out), lambda: dg.rmsnorm_bf16_backward(x, x, None, s, out),
                 lambda: dg.gemm_int8_nt_epilogue((q, s), (q, s), torch.empty((4, 4), device="cuda")),
                 lambda: dg.quantize_int8_rows(x), lambda: dg.moe_sort_masked(ids, 8, ids[0], ids),
                 lambda: dg.moe_dispatch_bf16(x, ids, out), lambda: dg.moe_combine_bf16(out, ids, x)):
        with pytest.raises(ValueError, match="not the current one"):
            call()


@pytest.mark.parametrize("t,h,stride", [(1, 256, 0), (3, 256, 264), (2, 1, 8)])
@pytest.mark.parametrize("weight", [BF16, F32, None])
@pytest.mark.parametrize("eps", [1e-6, 0, 1])
def test_native_arguments_are_the_binding_s(dg, t, h, stride, weight, eps):
    """What the native helper makes of a call's tensors is what the functions in Python behind it make."""
    say(f"native arguments {t}x{h}")
    x, r, w = inputs(t, h, True, weight, 11, stride)
    total, rstd = torch.empty_like(x), torch.empty(t, device="cuda")
    for args in ((x, (t, h), w, eps, r, total, rstd, 0), (x, (t, h), w, eps, None, None, None, 0)):
        assert dg._norm(*args) == dg._norm_of(*args)
    current = dg._current_device
    assert dg._matrix(x, "x", current) == dg._matrix_of(x, "x", current)
    if w is not None:
        assert dg._vector(w, h, 0, "w") == dg._vector_of(w, h, 0, "w")
    q = torch.zeros((t, h), dtype=torch.uint8, device="cuda")
    a = torch.zeros((2, t, h), dtype=FP8, device="cuda")
    rows = torch.zeros((t, 3), dtype=torch.int32, device="cuda")
    for b in (q, q.view(FP8)):
        assert dg._bytes8(b, (t, h), 0, "q") == dg._bytes8_of(b, (t, h), 0, "q")
        assert dg._layout(b, None, h, 0, "a") == dg._layout_of(b, None, h, 0, "a")
    assert dg._layout(a, None, h, 0, "a") == dg._layout_of(a, None, h, 0, "a") == (a.data_ptr(), 2 * t)
    assert dg._layout(rows, torch.int32, 3, 0, "a") == dg._layout_of(rows, torch.int32, 3, 0, "a")
    assert dg._slots(rows, t, 0) == dg._slots_of(rows, t, 0)


def test_native_arguments_refuse_as_the_binding_does(dg):
    """Every mismatch ends in the same error as without the native helper."""
    x, _, w = inputs(4, 256, False, F32, 12)
    q, rows = torch.zeros((4, 256), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    n = lambda **kw: tuple({**dict(x=x, shape=(4, 256), weight=w, eps=1e-6, residual=None, sum_out=None, rstd=None, dev=0),
                            **kw}.values())
    cases = [("_norm", n(weight=w[:255])), ("_norm", n(weight=w.to(torch.float16))), ("_norm", n(residual=x[:3])),
             ("_norm", n(sum_out=x.float())), ("_norm", n(rstd=w)), ("_norm", n(dev=1)), ("_norm", n(eps="1")),
             ("_norm", n(eps=1e39)), ("_norm", n(residual=x.t())), ("_norm", n(weight=w.cpu())), ("_norm", n(residual=3)),
             ("_matrix", (w, "x", dg._current_device)), ("_matrix", (x.cpu(), "x", dg._current_device)),
             ("_matrix", (x, "x", lambda: 5)), ("_vector", (w, 255, 0, "w")), ("_vector", (w.double(), 256, 0, "w")),
             ("_vector", (x, 256, 0, "w")), ("_bytes8", (x, (4, 256), 0, "q")), ("_bytes8", (q, (4, 255), 0, "q")),
             ("_bytes8", (q[:, ::2], (4, 128), 0, "q")), ("_layout", (q, None, 255, 0, "a")),
             ("_layout", (x, None, 256, 0, "a")), ("_layout", (x, F32, 256, 0, "a")), ("_layout", (w, F32, 256, 0, "a")),
             ("_slots", (rows, 3, 0)), ("_slots", (rows.long(), 4, 0)), ("_slots", (rows.t(), 2, 0)), ("_slots", (rows, 4, 1))]

    def outcome(f, args):
        try:
            return f(*args)
        except Exception as e:
            return type(e), str(e)

    refused = 0
    for name, args in cases:
        python = outcome(getattr(dg, name + "_of"), args)
        assert outcome(getattr(dg, name), args) == python, name
        refused += isinstance(python, tuple) and isinstance(python[0], type)
    assert refused == len(cases) - 1  # (an eps past fp32 packs as an infinity, which the library refuses)
    with pytest.raises(dg.DGError):
        dg.rmsnorm_bf16(x, w, torch.empty_like(x), 1e39)


@pytest.mark.parametrize("h", [1, 2, 3, 5, 7, 9, 15, 31, 33, 47, 63, 65, 130, 257, 513, 519, 1161, 4097, 8199])
@pytest.mark.parametrize("t,gap", [(3, 0), (3, 5), (70, 0), (800, 1)])
def test_rows_of_every_tail(dg, t, h, gap):
    """Rows that end 1 to 7 values past a multiple of 8, close to each other: nothing beside them is read or written."""
    say(f"norm tails {t}x{h} gap {gap}")
    x, r, w = inputs(t, h, True, BF16, 13, h + gap, 3)
    space = torch.full((t * (h + gap) + 8,), 7.0, dtype=BF16, device="cuda")
    out = space[4:4 + t * (h + gap)].view(t, h + gap)[:, :h]
    total, rstd = torch.empty((t, h), dtype=BF16, device="cuda"), torch.empty(t, device="cuda")
    dg.rmsnorm_bf16(x, w, out, 1e-6, r, total, rstd)
    z, _, y = ref64(x, r, w, 1e-6)
    within(out, y, (2.0 ** -8 + 2.0 ** -16) * y.abs(), "y")
    within(total, z, (2.0 ** -8 + 2.0 ** -24) * z.abs(), "sum")
    q, s = torch.full((t * h + 8,), 55, dtype=torch.int8, device="cuda"), torch.empty(t, device="cuda")
    dg.rmsnorm_quantize_int8(x, w, q[:t * h].view(t, h), s, 1e-6, r)
    se = s.to(F64)[:, None]
    within(q[:t * h].view(t, h).to(F64) * se, y, 0.5 * se + 2.0 ** -15 * y.abs(), "int8")
    assert (q[t * h:] == 55).all()
    dy = inputs(t, h, False, None, 14, h + gap, 1)[0]
    dw = torch.full((h + 8,), 9.0, device="cuda")
    back = torch.full_like(space, 7.0)
    dx = back[4:4 + t * (h + gap)].view(t, h + gap)[:, :h]
    dg.rmsnorm_bf16_backward(dy, x, w, rstd, dx, dw[:h], r)
    wx, bx, ww, bw = backward64(dy, x, w, rstd, r)
    within(dx, wx, bx, "dx")
    within(dw[:h], ww, bw, "dw")
    assert (dw[h:] == 9).all()
    for buf, rows in ((space, out), (back, dx)):
        rows.fill_(7.0)
        assert (buf == 7).all()


def test_offsets_past_32_bits(dg):
    """Rows two GB apart, forward and backward."""
    t, h, stride = 4, 1000, (1 << 30) + 8
    say("norm rows 2 GB apart")
    far = torch.zeros((t - 1) * stride + h, dtype=BF16, device="cuda").as_strided((t, h), (stride, 1))
    x, r, w = inputs(t, h, True, F32, 15)
    far.copy_(x)
    out, near = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(t, device="cuda")
    dg.rmsnorm_bf16(x, w, near, 1e-6, r, rstd=rstd)
    dg.rmsnorm_bf16(far, w, out, 1e-6, r)
    assert torch.equal(out, near)
    q, s, q2, s2 = (torch.empty(n, dtype=d, device="cuda") for n, d in (((t, h), torch.int8), (t, F32)) * 2)
    dg.rmsnorm_quantize_int8(x, w, q, s)
    dg.rmsnorm_quantize_int8(far, w, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    dx, dw, dw2 = torch.empty_like(x), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    dg.rmsnorm_bf16_backward(r, x, w, rstd, dx, dw)
    dg.rmsnorm_bf16_backward(r, far, w, rstd, out, dw2)
    assert torch.equal(out, dx) and torch.equal(dw, dw2)
    dg.rmsnorm_bf16(x, w, far, 1e-6, r)
    assert torch.equal(far, near)
    far.copy_(x)
    dg.rmsnorm_bf16_backward(r, x, w, rstd, far)
    assert torch.equal(far, dx)
