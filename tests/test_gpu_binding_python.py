"""The calls whose tensors are checked natively, with the Python functions that
stand in where the native helper is missing: the same results, the same refusals."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, I32, I8, FP8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.float8_e4m3fn
NAMES = ["_whole", "_rows", "_matrix", "_vector", "_bytes8", "_layout", "_slots", "_norm"]


@pytest.fixture(scope="module")
def dg():
    import moe_grouped_gemm_x128_amd as m
    return m


@pytest.fixture
def python(dg, monkeypatch):
    def use():
        for n in NAMES:
            monkeypatch.setattr(dg, n, getattr(dg, n + "_of"))
    return use


def everything(dg):
    """Every such call once on the same inputs; all they write."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    new = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device="cuda")
    t, h, e, k = 37, 512, 6, 2
    wide = rn(t, h + 24).to(BF16)
    x, r, w = wide[:, 8:8 + h], rn(t, h).to(BF16), rn(h)
    total, rstd, y = new(t, h), new(t, dtype=F32), new(t, h)
    out = [total, rstd, dg.rmsnorm_bf16(x, w, y, 1e-6, r, total, rstd)]
    q, s = new(t, h, dtype=FP8), new(t, h // 128, dtype=F32)
    out += dg.rmsnorm_quantize_fp8_1x128(x, w.to(BF16), q, s, 1, r)
    qp, sp = new(t, h, dtype=torch.uint8), new(t, 1, dtype=I32)
    out += dg.rmsnorm_quantize_fp8_1x128(x, None, qp, sp)
    a8 = dg.rmsnorm_quantize_int8(x, w, new(t, h, dtype=I8), new(t, dtype=F32))
    b8 = dg.quantize_int8_rows(rn(80, h))
    out += [*a8, *b8, dg.gemm_int8_nt_epilogue(a8, b8, new(t, 80), rn(80), "gelu", rn(t, 80).to(BF16), new(t, 80))]
    out += dg.rmsnorm_bf16_backward(y, total, w, rstd, new(t, h), new(h, dtype=F32), r)
    ids = torch.randint(-1, e, (t, k), generator=g, device="cuda").to(I32)
    m = dg.moe_sort_rows(t, k, e)
    mi, rows = dg.moe_sort_contiguous(ids, e, new(m, dtype=I32), new(t, k, dtype=I32), new(e, dtype=I32))
    mm, mrows = dg.moe_sort_masked(ids, 64, new(e, dtype=I32), new(t, k, dtype=I32))
    o = dg.moe_dispatch_bf16(y, rows, new(m, h), mi)
    a, sa = dg.moe_dispatch_fp8((q, s), mrows, (new(e, 64, h, dtype=FP8), new(e, 64, h // 128, dtype=F32)))
    weights = torch.rand((t, k), generator=g, device="cuda")
    out += [mi, rows, mm, mrows, o, a, sa, dg.moe_combine_bf16(o, rows, new(t, h), weights, r)]
    out += dg.moe_combine_bf16_backward(y, o, rows, weights, new(m, h), new(t, k, dtype=F32), mi)
    out.append(dg.moe_dispatch_bf16_backward(o, rows, new(t, h)))
    return [v.view(torch.uint8) if v.dtype == FP8 else v for v in out]


def test_same_results(dg, python):
    native = everything(dg)
    python()
    for i, (a, b) in enumerate(zip(native, everything(dg))):
        assert torch.equal(a, b), i


def test_same_refusals(dg):
    x = torch.zeros((4, 256), dtype=BF16, device="cuda")
    cases = [(x, BF16, (4, 256), 0), (x, F32, (4, 256), 0), (x, BF16, (4, 255), 0), (x, BF16, (1024,), 0),
             (x, BF16, (4, 256), 1), (x.t(), BF16, (256, 4), 0), (x[:, ::2], BF16, (4, 128), 0), (x[:, :8], BF16, (4, 8), 0),
             (x[:1].expand(4, 256), BF16, (4, 256), 0), (x[:1, ::2][:, :1], BF16, (1, 1), 0), (x.cpu(), BF16, (4, 256), 0),
             (x[0], BF16, (256,), 0), (3, BF16, (4, 256), 0)]

    def outcome(f, args):
        try:
            return f(*args, "t")
        except Exception as e:
            return type(e), str(e)

    for name in ("_whole", "_rows"):
        for i, args in enumerate(cases):
            assert outcome(getattr(dg, name), args) == outcome(getattr(dg, name + "_of"), args), (name, i)
