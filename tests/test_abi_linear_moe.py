"""Refusals of the linear-layer and few-token MoE entry points on the CPU: bad
arguments come back as a status before anything touches the GPU (the pointers
are made-up addresses that a call which got further would have to read)."""
from __future__ import annotations

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_grouped_gemm_x128_amd", "libdg_mi355x.so")

INVALID, UNSUPPORTED = 1, 2
P = 0x10000  # a 16-byte aligned address
BF16, F32 = 0, 1


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_type", ctypes.c_int), ("activation", ctypes.c_int),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
                ("pre", ctypes.c_void_p), ("ld_pre", ctypes.c_int64)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import subprocess
        import sys
        subprocess.run([sys.executable, os.path.join(ROOT, "moe_grouped_gemm_x128_amd", "build.py")], check=True)
    L = ctypes.CDLL(LIB)
    vp, i, l, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    L.dg_gemm_bf16_nt_epilogue.argtypes = [vp, l, vp, l, vp, l, i, vp, i, i, i, vp]
    L.dg_gemm_fp8_nt_epilogue.argtypes = [vp, vp, vp, vp, vp, l, i, vp, i, i, i, vp]
    L.dg_gemm_bf16_nt_epilogue_backward.argtypes = [vp, l, vp, l, vp, l, vp, l, i, vp, l, vp, l, vp, vp, i, i, i, vp]
    L.dg_gemm_bf16_nt_epilogue_backward_workspace.argtypes = [i, i, ctypes.POINTER(l)]
    L.dg_moe_few_tokens_fp8.argtypes = [vp] * 11 + [i] * 7 + [f, vp]
    L.dg_moe_few_tokens_bf16.argtypes = [vp] * 9 + [i] * 7 + [f, vp]
    return L


def epilogue(**kw):
    e = Epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def forward(lib, fp8=False, a=P, b=P, c=P, lda=256, ldb=256, ldc=100, ct=BF16, e=None, m=10, n=100, k=256, sa=P, sb=P):
    ep = None if e is None else ctypes.addressof(e)
    if fp8:
        return lib.dg_gemm_fp8_nt_epilogue(a, sa, b, sb, c, ldc, ct, ep, m, n, k, None)
    return lib.dg_gemm_bf16_nt_epilogue(a, lda, b, ldb, c, ldc, ct, ep, m, n, k, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(a=None), dict(b=None), dict(c=None), dict(m=0), dict(n=-1), dict(k=0),
                                dict(ldc=99), dict(ct=2), dict(e=epilogue(activation=5)),
                                dict(e=epilogue(activation=-1)), dict(e=epilogue(bias=P, bias_type=7)),
                                dict(e=epilogue(residual=P, ld_residual=99)), dict(e=epilogue(pre=P, ld_pre=1))])
def test_forward_invalid(lib, fp8, kw):
    assert forward(lib, fp8, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(lda=255), dict(ldb=8)])
def test_forward_bf16_rows_overlap(lib, kw):
    assert forward(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(sa=None), dict(sb=None)])
def test_forward_fp8_without_scales(lib, kw):
    assert forward(lib, True, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(k=252), dict(a=P + 8), dict(b=P + 2), dict(lda=260), dict(ldb=1 << 23, k=256),
                                dict(c=P + 1), dict(ct=F32, c=P + 2), dict(ldc=(1 << 20) + 1),
                                dict(k=(1 << 22) + 8, lda=(1 << 22) + 8, ldb=(1 << 22) + 8),
                                dict(e=epilogue(residual=P + 1, ld_residual=100)),
                                dict(e=epilogue(bias=P + 2, bias_type=F32)),
                                dict(e=epilogue(pre=P, ld_pre=1 << 21))])
def test_forward_bf16_unsupported(lib, kw):
    assert forward(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(k=200), dict(a=P + 8), dict(b=P + 4), dict(sa=P + 2), dict(sb=P + 1),
                                dict(c=P + 1), dict(k=(1 << 22) + 128)])
def test_forward_fp8_unsupported(lib, kw):
    assert forward(lib, True, **kw) == UNSUPPORTED


def backward(lib, dc=P, lddc=100, a=P, lda=256, b=P, ldb=256, pre=P, ldp=100, act=4, da=P, ldda=256, db=P, lddb=256,
             dbias=P, ws=P, m=10, n=100, k=256):
    return lib.dg_gemm_bf16_nt_epilogue_backward(dc, lddc, a, lda, b, ldb, pre, ldp, act, da, ldda, db, lddb, dbias,
                                                 ws, m, n, k, None)


@pytest.mark.parametrize("kw", [dict(dc=None), dict(lddc=99), dict(a=None), dict(b=None), dict(lda=255), dict(ldb=0),
                                dict(pre=None), dict(ldp=99), dict(act=5), dict(act=-1), dict(ldda=255), dict(lddb=1),
                                dict(ws=None), dict(m=0), dict(n=0), dict(k=-8)])
def test_backward_invalid(lib, kw):
    assert backward(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(a=P + 2), dict(b=P + 8), dict(lda=260), dict(ws=P + 8), dict(da=P + 1),
                                dict(db=P + 1), dict(dbias=P + 2), dict(k=250, lda=256, ldb=256)])
def test_backward_unsupported(lib, kw):
    assert backward(lib, **kw) == UNSUPPORTED


def test_backward_workspace(lib):
    need = ctypes.c_int64()
    assert lib.dg_gemm_bf16_nt_epilogue_backward_workspace(0, 4, ctypes.byref(need)) == INVALID
    assert lib.dg_gemm_bf16_nt_epilogue_backward_workspace(4, 4, None) == INVALID
    last = 0
    for m, n in ((1, 1), (17, 9), (517, 1161), (4096, 7168)):
        assert lib.dg_gemm_bf16_nt_epilogue_backward_workspace(m, n, ctypes.byref(need)) == 0
        assert need.value >= 2 * m * n + 4 * n and need.value > last
        last = need.value


def moe(lib, fp8=True, x=P, logits=P, ids=P, weights=P, w13=P, s13=P, w2=P, s2=P, residual=None, y=P, ws=P, t=3, h=256,
        i=128, e=4, k=2, scoring=0, renorm=1, scale=1.0):
    tail = (residual, y, ws, t, h, i, e, k, scoring, renorm, scale, None)
    if fp8:
        return lib.dg_moe_few_tokens_fp8(x, logits, ids, weights, w13, s13, w2, s2, *tail)
    return lib.dg_moe_few_tokens_bf16(x, logits, ids, weights, w13, w2, *tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(x=None), dict(ids=None), dict(weights=None), dict(w13=None), dict(w2=None),
                                dict(y=None), dict(ws=None), dict(t=0), dict(h=0), dict(i=-128), dict(e=0), dict(k=0),
                                dict(scoring=2), dict(scoring=-1), dict(k=5)])
def test_moe_invalid(lib, fp8, kw):
    assert moe(lib, fp8, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(s13=None), dict(s2=None)])
def test_moe_fp8_without_scales(lib, kw):
    assert moe(lib, True, **kw) == INVALID


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(t=65), dict(h=200), dict(i=64), dict(e=513), dict(e=32, k=17), dict(x=P + 8),
                                dict(w13=P + 8), dict(w2=P + 4), dict(y=P + 4), dict(residual=P + 2), dict(ws=P + 8),
                                dict(ids=P + 2), dict(weights=P + 1), dict(logits=P + 2), dict(h=(1 << 20) + 128)])
def test_moe_unsupported(lib, fp8, kw):
    assert moe(lib, fp8, **kw) == UNSUPPORTED
