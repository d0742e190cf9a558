"""Refusals of the norm, the sorted-token and the INT8 entry points on the CPU: a
bad argument comes back as a status before anything touches the GPU (the
pointers are made-up addresses that a call which got further would have to
read)."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

from tests.test_abi_linear_moe import BF16, F32, INVALID, UNSUPPORTED, P, epilogue, lib as base_lib  # noqa: F401

OK, NONE = 0, None
vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class Norm(ctypes.Structure):
    _fields_ = [("x", vp), ("ld_x", i64), ("residual", vp), ("ld_residual", i64), ("weight", vp), ("weight_type", i32),
                ("eps", f32), ("sum", vp), ("ld_sum", i64), ("rstd", vp)]


@pytest.fixture(scope="module")
def lib(base_lib):  # noqa: F811
    L = base_lib
    L.dg_rmsnorm_bf16.argtypes = [vp, vp, i64, i32, i32, vp]
    for f in ("dg_rmsnorm_quantize_fp8_1x128", "dg_rmsnorm_quantize_fp8_1x128_ue8m0", "dg_rmsnorm_quantize_int8"):
        getattr(L, f).argtypes = [vp, vp, vp, i32, i32, vp]
    L.dg_rmsnorm_bf16_backward.argtypes = [vp, i64, vp, i64, vp, i32, vp, vp, i64, vp, i64, vp, vp, i32, i32, vp]
    L.dg_rmsnorm_bf16_backward_workspace.argtypes = [i32, i32, ctypes.POINTER(i64)]
    L.dg_moe_sort_contiguous.argtypes = [vp] * 5 + [i32] * 4 + [vp]
    L.dg_moe_sort_masked.argtypes = [vp] * 4 + [i32] * 4 + [vp]
    L.dg_moe_sort_workspace.argtypes = [i32, i32, i32, ctypes.POINTER(i64)]
    L.dg_moe_dispatch_bf16.argtypes = [vp, i64, vp, vp, vp, i32, i32, i32, i64, vp]
    for f in ("dg_moe_dispatch_fp8", "dg_moe_dispatch_fp8_ue8m0"):
        getattr(L, f).argtypes = [vp] * 6 + [i32] * 3 + [i64, vp]
    L.dg_moe_combine_bf16.argtypes = [vp, vp, vp, vp, i64, vp, i64, i32, i32, i32, i64, vp]
    L.dg_moe_combine_bf16_backward.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, vp]
    L.dg_gemm_int8_nt_epilogue.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i32, vp, i32, i32, i32, vp]
    L.dg_quantize_int8_rows.argtypes = [vp, i64, i32, vp, vp, i32, i32, vp]
    return L


OUTS = ["bf16", "fp8", "ue8m0", "int8"]


def norm(lib, out="bf16", y=P, s=P, ld_y=256, t=3, h=256, null=False, **kw):
    a = dict(x=P, ld_x=256, weight=P, weight_type=BF16, eps=1e-6)
    a.update(kw)
    n = Norm()
    for k, v in a.items():
        setattr(n, k, v)
    p = None if null else ctypes.addressof(n)
    if out == "bf16":
        return lib.dg_rmsnorm_bf16(p, y, ld_y, t, h, None)
    fn = {"fp8": lib.dg_rmsnorm_quantize_fp8_1x128, "ue8m0": lib.dg_rmsnorm_quantize_fp8_1x128_ue8m0,
          "int8": lib.dg_rmsnorm_quantize_int8}[out]
    return fn(p, y, s, t, h, None)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("kw", [dict(null=True), dict(x=NONE), dict(y=NONE), dict(t=0), dict(t=-4), dict(h=0),
                                dict(ld_x=255), dict(residual=P, ld_residual=128), dict(sum=P, ld_sum=0),
                                dict(weight_type=2), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))])
def test_norm_invalid(lib, out, kw):
    assert norm(lib, out, **kw) == INVALID


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("kw", [dict(x=P + 1), dict(residual=P + 1, ld_residual=256), dict(sum=P + 1, ld_sum=256),
                                dict(weight=P + 1), dict(weight=P + 2, weight_type=F32), dict(rstd=P + 2),
                                dict(h=16385, ld_x=16385, ld_y=16385), dict(ld_x=1 << 41)])
def test_norm_unsupported(lib, out, kw):
    assert norm(lib, out, **kw) == UNSUPPORTED


@pytest.mark.parametrize("out", OUTS[1:])
@pytest.mark.parametrize("s", [NONE, P + 2])
def test_norm_scales(lib, out, s):
    assert norm(lib, out, s=s) == (INVALID if s is None else UNSUPPORTED)


@pytest.mark.parametrize("kw", [dict(ld_y=255), dict(y=P + 1)])
def test_norm_bf16_output(lib, kw):
    assert norm(lib, **kw) == (INVALID if "ld_y" in kw else UNSUPPORTED)


@pytest.mark.parametrize("out", ["fp8", "ue8m0"])
@pytest.mark.parametrize("kw", [dict(h=200), dict(h=64), dict(y=P + 4)])
def test_norm_fp8_groups(lib, out, kw):
    assert norm(lib, out, **kw) == UNSUPPORTED


def backward(lib, dy=P, lddy=256, z=P, ldz=256, w=P, wt=F32, rstd=P, dsum=P, ldds=256, dx=P, lddx=256, dw=P, ws=P, t=3,
             h=256):
    return lib.dg_rmsnorm_bf16_backward(dy, lddy, z, ldz, w, wt, rstd, dsum, ldds, dx, lddx, dw, ws, t, h, None)


@pytest.mark.parametrize("kw", [dict(dy=NONE), dict(z=NONE), dict(rstd=NONE), dict(t=0), dict(h=-1), dict(lddy=255),
                                dict(ldz=1), dict(lddx=128), dict(ldds=255), dict(wt=3), dict(ws=NONE, t=5000)])
def test_norm_backward_invalid(lib, kw):
    assert backward(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dy=P + 1), dict(z=P + 1), dict(rstd=P + 1), dict(dsum=P + 1), dict(dx=P + 1),
                                dict(dw=P + 2), dict(ws=P + 4, t=5000), dict(w=P + 2),
                                dict(h=1 << 15, lddy=1 << 15, ldz=1 << 15, ldds=1 << 15, lddx=1 << 15)])
def test_norm_backward_unsupported(lib, kw):
    assert backward(lib, **kw) == UNSUPPORTED


def test_norm_backward_of_nothing(lib):
    """Neither gradient is asked for: nothing is done, and what only they need is not looked at."""
    assert backward(lib, dx=NONE, dw=NONE, ws=NONE, lddx=0, dsum=P + 1) == OK


def test_norm_backward_workspace(lib):
    need = i64()
    assert lib.dg_rmsnorm_bf16_backward_workspace(0, 4, ctypes.byref(need)) == INVALID
    assert lib.dg_rmsnorm_bf16_backward_workspace(4, -1, ctypes.byref(need)) == INVALID
    assert lib.dg_rmsnorm_bf16_backward_workspace(4, 4, None) == INVALID
    assert lib.dg_rmsnorm_bf16_backward_workspace(3, 100, ctypes.byref(need)) == OK and need.value == 0
    last = 0
    for t, h in ((5000, 1), (6000, 1000), (600000, 16384)):
        assert lib.dg_rmsnorm_bf16_backward_workspace(t, h, ctypes.byref(need)) == OK
        assert need.value >= 4 * h and need.value > last
        last = need.value


def sort(lib, masked, ids=P, first=P, rows=P, counts=P, ws=P, t=5, k=2, e=4, m=256):
    if masked:
        return lib.dg_moe_sort_masked(ids, first, rows, ws, t, k, e, m, None)
    return lib.dg_moe_sort_contiguous(ids, first, rows, counts, ws, t, k, e, m, None)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("kw", [dict(ids=NONE), dict(first=NONE), dict(rows=NONE), dict(t=0), dict(k=0), dict(e=0),
                                dict(e=-3), dict(m=0), dict(m=-128), dict(t=100000, ws=NONE)])
def test_sort_invalid(lib, masked, kw):
    assert sort(lib, masked, **kw) == INVALID


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("kw", [dict(k=17), dict(e=1025), dict(t=1 << 23), dict(ids=P + 2), dict(first=P + 1),
                                dict(rows=P + 2), dict(t=100000, ws=P + 2), dict(t=1 << 30, k=16)])
def test_sort_unsupported(lib, masked, kw):
    assert sort(lib, masked, **kw) == UNSUPPORTED


def test_sort_layout_limits(lib):
    assert sort(lib, False, m=200) == UNSUPPORTED
    assert sort(lib, False, counts=P + 2) == UNSUPPORTED
    assert sort(lib, True, e=1024, m=1 << 21) == UNSUPPORTED
    assert sort(lib, True, e=1, m=(1 << 31) - 5) == UNSUPPORTED


def test_sort_workspace(lib):
    need = i64()
    assert lib.dg_moe_sort_workspace(1, 1, 1, None) == INVALID
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0)):
        assert lib.dg_moe_sort_workspace(*bad, ctypes.byref(need)) == INVALID
    for bad in ((1, 17, 4), (1, 1, 1025), (1 << 23, 2, 4)):
        assert lib.dg_moe_sort_workspace(*bad, ctypes.byref(need)) == UNSUPPORTED
    assert lib.dg_moe_sort_workspace(1, 8, 256, ctypes.byref(need)) == OK and need.value == 0
    assert lib.dg_moe_sort_workspace(1 << 23, 1, 1024, ctypes.byref(need)) == OK and need.value >= 4096


def dispatch(lib, fp8, x=P, s=P, ldx=256, rows=P, mi=P, a=P, sa=P, t=5, k=2, h=256, m=256):
    if fp8:
        fn = lib.dg_moe_dispatch_fp8_ue8m0 if fp8 == "ue8m0" else lib.dg_moe_dispatch_fp8
        return fn(x, s, rows, mi, a, sa, t, k, h, m, None)
    return lib.dg_moe_dispatch_bf16(x, ldx, rows, mi, a, t, k, h, m, None)


@pytest.mark.parametrize("fp8", [None, "f32", "ue8m0"])
@pytest.mark.parametrize("kw", [dict(x=NONE), dict(rows=NONE), dict(a=NONE), dict(t=0), dict(k=-1), dict(h=0), dict(m=0)])
def test_dispatch_invalid(lib, fp8, kw):
    assert dispatch(lib, fp8, **kw) == INVALID


@pytest.mark.parametrize("fp8", [None, "f32", "ue8m0"])
@pytest.mark.parametrize("kw", [dict(k=17), dict(x=P + 8), dict(a=P + 8), dict(rows=P + 2), dict(mi=P + 2), dict(m=200),
                                dict(h=252), dict(h=(1 << 20) + 128, ldx=1 << 21), dict(m=1 << 31), dict(t=1 << 23)])
def test_dispatch_unsupported(lib, fp8, kw):
    assert dispatch(lib, fp8, **kw) == UNSUPPORTED


def test_dispatch_scales_and_strides(lib):
    for fp8 in ("f32", "ue8m0"):
        assert dispatch(lib, fp8, s=NONE) == INVALID and dispatch(lib, fp8, sa=NONE) == INVALID
        assert dispatch(lib, fp8, s=P + 2) == UNSUPPORTED and dispatch(lib, fp8, sa=P + 1) == UNSUPPORTED
    assert dispatch(lib, None, ldx=255) == INVALID
    assert dispatch(lib, None, ldx=260) == UNSUPPORTED


def combine(lib, o=P, rows=P, w=P, res=P, ldr=256, y=P, ldy=256, t=5, k=2, h=256, m=256):
    return lib.dg_moe_combine_bf16(o, rows, w, res, ldr, y, ldy, t, k, h, m, None)


@pytest.mark.parametrize("kw", [dict(o=NONE), dict(rows=NONE), dict(y=NONE), dict(ldy=255), dict(ldr=8), dict(t=0),
                                dict(k=0), dict(h=0), dict(m=0)])
def test_combine_invalid(lib, kw):
    assert combine(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(o=P + 8), dict(y=P + 2), dict(res=P + 8), dict(w=P + 2), dict(ldy=260),
                                dict(ldr=257), dict(h=252), dict(k=17), dict(m=1 << 31), dict(rows=P + 1)])
def test_combine_unsupported(lib, kw):
    assert combine(lib, **kw) == UNSUPPORTED


def combine_backward(lib, dy=P, lddy=256, o=P, rows=P, w=P, mi=P, do=P, dw=P, t=5, k=2, h=256, m=256):
    return lib.dg_moe_combine_bf16_backward(dy, lddy, o, rows, w, mi, do, dw, t, k, h, m, None)


@pytest.mark.parametrize("kw", [dict(dy=NONE), dict(o=NONE), dict(rows=NONE), dict(lddy=255), dict(t=0), dict(k=0),
                                dict(h=0), dict(m=0)])
def test_combine_backward_invalid(lib, kw):
    assert combine_backward(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dy=P + 2), dict(lddy=257), dict(o=P + 8), dict(do=P + 8), dict(w=P + 1),
                                dict(dw=P + 2), dict(mi=P + 2), dict(m=200), dict(h=250), dict(k=17)])
def test_combine_backward_unsupported(lib, kw):
    assert combine_backward(lib, **kw) == UNSUPPORTED


def test_combine_backward_of_nothing(lib):
    assert combine_backward(lib, do=NONE, dw=NONE, o=NONE) == OK


def int8(lib, a=P, lda=256, sa=P, b=P, ldb=256, sb=P, c=P, ldc=100, ct=BF16, e=None, m=10, n=100, k=256):
    ep = None if e is None else ctypes.addressof(e)
    return lib.dg_gemm_int8_nt_epilogue(a, lda, sa, b, ldb, sb, c, ldc, ct, ep, m, n, k, None)


@pytest.mark.parametrize("kw", [dict(a=NONE), dict(sa=NONE), dict(b=NONE), dict(sb=NONE), dict(c=NONE), dict(m=0),
                                dict(n=0), dict(k=-16), dict(lda=255), dict(ldb=16), dict(ldc=99), dict(ct=2),
                                dict(e=epilogue(activation=5)), dict(e=epilogue(bias=P, bias_type=7)),
                                dict(e=epilogue(residual=P, ld_residual=99)), dict(e=epilogue(pre=P, ld_pre=1))])
def test_int8_invalid(lib, kw):
    assert int8(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(k=248), dict(a=P + 8), dict(b=P + 4), dict(lda=264), dict(ldb=257),
                                dict(sa=P + 2), dict(sb=P + 1), dict(c=P + 1), dict(ct=F32, c=P + 2),
                                dict(k=1 << 17, lda=1 << 17, ldb=1 << 17), dict(lda=(1 << 22) + 16),
                                dict(ldc=(1 << 20) + 1), dict(e=epilogue(bias=P + 2, bias_type=F32))])
def test_int8_unsupported(lib, kw):
    assert int8(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw,want", [(dict(x=NONE), INVALID), (dict(q=NONE), INVALID), (dict(s=NONE), INVALID),
                                     (dict(m=0), INVALID), (dict(k=0), INVALID), (dict(ld=99), INVALID),
                                     (dict(kind=2), INVALID), (dict(x=P + 1), UNSUPPORTED), (dict(s=P + 2), UNSUPPORTED),
                                     (dict(x=P + 2, kind=F32), UNSUPPORTED)])
def test_quantize_int8(lib, kw, want):
    a = dict(x=P, ld=100, kind=BF16, q=P, s=P, m=4, k=100)
    a.update(kw)
    assert lib.dg_quantize_int8_rows(a["x"], a["ld"], a["kind"], a["q"], a["s"], a["m"], a["k"], None) == want


def test_quantize_int8_of_too_long_rows(lib):
    """Column numbers and the step past the last one stay in 32 bits."""
    k = (1 << 30) + 1
    assert lib.dg_quantize_int8_rows(P, k, BF16, P, P, 1, k, None) == UNSUPPORTED


def test_binding_wants_the_gpu():
    """Tensors on the host are refused by every call of the binding."""
    import moe_grouped_gemm_x128_amd as dg
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256), dtype=torch.int8), torch.zeros(4)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    mi = torch.zeros(128, dtype=torch.int32)
    a = torch.zeros((128, 256), dtype=torch.bfloat16)
    for call in (lambda: dg.rmsnorm_bf16(x, None, x), lambda: dg.rmsnorm_quantize_int8(x, None, q, s),
                 lambda: dg.rmsnorm_bf16_backward(x, x, None, s, x),
                 lambda: dg.rmsnorm_quantize_fp8_1x128(x, None, q.view(torch.uint8), torch.zeros((4, 2))),
                 lambda: dg.gemm_int8_nt_epilogue((q, s), (q, s), torch.zeros((4, 4))),
                 lambda: dg.quantize_int8_rows(x), lambda: dg.moe_sort_contiguous(ids, 2, mi, ids),
                 lambda: dg.moe_sort_masked(ids, 8, mi, ids), lambda: dg.moe_dispatch_bf16(x, ids, a),
                 lambda: dg.moe_dispatch_fp8((q.view(torch.uint8), torch.zeros((4, 2))), ids,
                                             (a.view(torch.uint8)[:, :256], torch.zeros((128, 2)))),
                 lambda: dg.moe_combine_bf16(a, ids, x), lambda: dg.moe_combine_bf16_backward(x, a, ids, None, a)):
        with pytest.raises(ValueError):
            call()


def test_rows_that_hold_any_routing():
    """moe_sort_rows against the worst routing: as many experts as can have one row more than a multiple of 128."""
    import moe_grouped_gemm_x128_amd as dg
    for t, k, e in ((1, 1, 1), (1, 8, 256), (64, 8, 32), (777, 6, 24), (8192, 8, 256)):
        slots, worst = t * k, 0
        for used in range(1, min(e, slots) + 1):  # every used expert but the first has one row of its last block
            first = slots - (used - 1)
            worst = max(worst, (first + 127) // 128 * 128 + (used - 1) * 128)
        assert dg.moe_sort_rows(t, k, e) >= worst and dg.moe_sort_rows(t, k, e) % 128 == 0
