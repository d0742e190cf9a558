"""Python binding of the MI355X FP8 fine-grained-scaled NT GEMM library.

Argument marshalling only: every function below checks tensor dtypes, shapes
and devices, then calls the C ABI (include/dg.h) of libdg_mi355x.so with raw
device pointers and the current HIP stream.  All arithmetic runs in the HIP
kernels; there is no CPU path.  If the library has not been built the import
fails loudly (build it with `python moe_grouped_gemm_x128_amd/build.py`).

The C-named functions mirror the C entry points one to one.  The
`*_fp8_fp8_*` names follow the call style of the DeepGEMM pages' usage example
(operands passed as (fp8 tensor, fp32 scale tensor) tuples, output tensor
preallocated by the caller).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import warnings

import torch  # loads torch's HIP runtime first, so the library binds to it

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg_mi355x.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python moe_grouped_gemm_x128_amd/build.py); there is no fallback path")

_lib = ctypes.CDLL(LIB_PATH)

try:  # the binding's checks of tensors, natively: not needed, but 2.5 us of a call
    from . import _tensors
    if getattr(_tensors, "built_with", None) != str(torch.__version__):
        raise ImportError(f"it was built with torch {getattr(_tensors, 'built_with', 'of another version')}")
except ImportError as _e:
    _tensors = None
    warnings.warn(f"the binding's native helper cannot be used ({_e}), so small calls take longer; "
                  "python moe_grouped_gemm_x128_amd/build.py builds it", RuntimeWarning)

_vp, _i32 = ctypes.c_void_p, ctypes.c_int
_lib.dg_gemm_fp8_nt.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_grouped_fp8_contiguous.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_grouped_fp8_contiguous_swiglu.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_grouped_fp8_masked.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_grouped_fp8_masked_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_wgrad_fp8_nt.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_k_grouped_wgrad_fp8_nt.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_gemm_fp8_nt_ue8m0.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_gemm_fp8_nt_ue8m0_packed.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_grouped_fp8_contiguous_ue8m0_packed.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_grouped_fp8_masked_ue8m0_packed.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_gemm_bf16_nt.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_grouped_bf16_contiguous.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_grouped_bf16_masked.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp]
_lib.dg_quantize_fp8_1x128.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
_lib.dg_quantize_fp8_128x128.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
_lib.dg_quantize_fp8_1x128_transposed.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
_lib.dg_quantize_fp8_1x128_ue8m0.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
_lib.dg_quantize_fp8_128x128_ue8m0.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
_lib.dg_swiglu_quantize_fp8_1x128.argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
for _f in ("dg_gemm_fp8_nt", "dg_grouped_fp8_contiguous", "dg_grouped_fp8_contiguous_swiglu", "dg_grouped_fp8_masked", "dg_grouped_fp8_masked_noalloc",
           "dg_wgrad_fp8_nt", "dg_k_grouped_wgrad_fp8_nt", "dg_gemm_fp8_nt_ue8m0", "dg_gemm_fp8_nt_ue8m0_packed", "dg_grouped_fp8_contiguous_ue8m0_packed",
           "dg_grouped_fp8_masked_ue8m0_packed", "dg_gemm_bf16_nt", "dg_grouped_bf16_contiguous", "dg_grouped_bf16_masked", "dg_quantize_fp8_1x128",
           "dg_quantize_fp8_128x128", "dg_quantize_fp8_1x128_transposed", "dg_swiglu_quantize_fp8_1x128",
           "dg_quantize_fp8_1x128_ue8m0", "dg_quantize_fp8_128x128_ue8m0"):
    getattr(_lib, _f).restype = ctypes.c_int
_f32c, _i64 = ctypes.c_float, ctypes.c_int64


class _Epilogue(ctypes.Structure):
    _fields_ = [("bias", _vp), ("bias_type", _i32), ("activation", _i32), ("residual", _vp), ("ld_residual", _i64),
                ("pre", _vp), ("ld_pre", _i64)]


_lib.dg_gemm_bf16_nt_epilogue.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i32, _i32, _i32, _vp]
_lib.dg_gemm_bf16_nt_epilogue.restype = ctypes.c_int
_lib.dg_gemm_fp8_nt_epilogue.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i32, _vp, _i32, _i32, _i32, _vp]
_lib.dg_gemm_fp8_nt_epilogue.restype = ctypes.c_int
_lib.dg_gemm_bf16_nt_epilogue_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _i64, _vp,
                                                   _i64, _vp, _vp, _i32, _i32, _i32, _vp]
_lib.dg_gemm_bf16_nt_epilogue_backward.restype = ctypes.c_int
_lib.dg_gemm_bf16_nt_epilogue_backward_workspace.argtypes = [_i32, _i32, ctypes.POINTER(_i64)]
_lib.dg_gemm_bf16_nt_epilogue_backward_workspace.restype = ctypes.c_int
_lib.dg_moe_few_tokens_fp8.argtypes = [_vp] * 11 + [_i32] * 7 + [_f32c, _vp]
_lib.dg_moe_few_tokens_fp8.restype = ctypes.c_int
_lib.dg_moe_few_tokens_bf16.argtypes = [_vp] * 9 + [_i32] * 7 + [_f32c, _vp]
_lib.dg_moe_few_tokens_bf16.restype = ctypes.c_int
_lib.dg_rmsnorm_bf16.argtypes = [_vp, _vp, _i64, _i32, _i32, _vp]
_lib.dg_rmsnorm_bf16_backward.argtypes = [_vp, _i64, _vp, _i64, _vp, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i32,
                                          _i32, _vp]
_lib.dg_rmsnorm_bf16_backward_workspace.argtypes = [_i32, _i32, ctypes.POINTER(_i64)]
_lib.dg_moe_sort_contiguous.argtypes = [_vp] * 5 + [_i32] * 4 + [_vp]
_lib.dg_moe_sort_masked.argtypes = [_vp] * 4 + [_i32] * 4 + [_vp]
_lib.dg_moe_sort_workspace.argtypes = [_i32, _i32, _i32, ctypes.POINTER(_i64)]
_lib.dg_moe_dispatch_bf16.argtypes = [_vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _vp]
_lib.dg_moe_combine_bf16.argtypes = [_vp, _vp, _vp, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _i64, _vp]
_lib.dg_moe_combine_bf16_backward.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i64, _vp]
_lib.dg_gemm_int8_nt_epilogue.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i32, _vp, _i32, _i32, _i32, _vp]
_lib.dg_quantize_int8_rows.argtypes = [_vp, _i64, _i32, _vp, _vp, _i32, _i32, _vp]
for _f in ("dg_rmsnorm_quantize_fp8_1x128", "dg_rmsnorm_quantize_fp8_1x128_ue8m0", "dg_rmsnorm_quantize_int8"):
    getattr(_lib, _f).argtypes = [_vp, _vp, _vp, _i32, _i32, _vp]
for _f in ("dg_moe_dispatch_fp8", "dg_moe_dispatch_fp8_ue8m0"):
    getattr(_lib, _f).argtypes = [_vp] * 6 + [_i32] * 3 + [_i64, _vp]
for _f in ("dg_rmsnorm_bf16", "dg_rmsnorm_quantize_fp8_1x128", "dg_rmsnorm_quantize_fp8_1x128_ue8m0",
           "dg_rmsnorm_quantize_int8", "dg_rmsnorm_bf16_backward", "dg_rmsnorm_bf16_backward_workspace",
           "dg_moe_sort_contiguous", "dg_moe_sort_masked", "dg_moe_sort_workspace", "dg_moe_dispatch_bf16",
           "dg_moe_dispatch_fp8", "dg_moe_dispatch_fp8_ue8m0", "dg_moe_combine_bf16", "dg_moe_combine_bf16_backward",
           "dg_gemm_int8_nt_epilogue", "dg_quantize_int8_rows"):
    getattr(_lib, _f).restype = ctypes.c_int
_lib.dg_status_string.argtypes = [ctypes.c_int]
_lib.dg_status_string.restype = ctypes.c_char_p
_lib.dg_version.restype = ctypes.c_int


class TileConfig(ctypes.Structure):
    _fields_ = [("block_m", ctypes.c_int), ("block_n", ctypes.c_int), ("waves_m", ctypes.c_int),
                ("waves_n", ctypes.c_int), ("tiles", ctypes.c_int), ("grid", ctypes.c_int),
                ("k_splits", ctypes.c_int), ("kernel", ctypes.c_int)]


_lib.dg_select_config.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(TileConfig)]
_lib.dg_select_config.restype = ctypes.c_int

(KIND_DENSE, KIND_CONTIGUOUS, KIND_MASKED, KIND_WGRAD, KIND_K_GROUPED_WGRAD, KIND_DENSE_POW2, KIND_BF16,
 KIND_CONTIGUOUS_SWIGLU, KIND_CONTIGUOUS_POW2, KIND_MASKED_POW2, KIND_CONTIGUOUS_BF16, KIND_MASKED_BF16) = range(12)
FP8 = torch.float8_e4m3fn


class DGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.dg_status_string(status).decode()
        super().__init__(f"{where}: status {status} ({msg})")


def _check(status: int, where: str):
    if status != 0:
        raise DGError(status, where)


# The current stream's raw handle without building a torch Stream object
# (a few microseconds per call otherwise, which small GEMMs would feel).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return t.data_ptr()


def _dev(*ts):
    if not ts[0].is_cuda:
        raise ValueError("tensors must live on the GPU")
    dev = ts[0].get_device()
    for t in ts:
        if not t.is_cuda or t.get_device() != dev:
            raise ValueError("all tensors must be on the same device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _fp8(t, name):
    if t.dtype not in (FP8, torch.uint8):
        raise TypeError(f"{name} must be float8_e4m3fn (or its uint8 bytes), got {t.dtype}")


def _f32(t, name):
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")


def _bf16(t, name):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def version() -> int:
    return _lib.dg_version()


def select_config(kind: int, m: int, n: int, k: int, num_groups: int = 1, num_cus: int = 256) -> dict:
    """Tile configuration the heuristic picks (host only, no GPU needed)."""
    cfg = TileConfig()
    _check(_lib.dg_select_config(kind, m, n, k, num_groups, num_cus, ctypes.byref(cfg)),
           "dg_select_config")
    return {f: getattr(cfg, f) for f, _ in TileConfig._fields_}


# ---------------------------------------------------------------- C names ---

def dg_gemm_fp8_nt(a, sa, b, sb, c):
    """C[M,N] bf16 = fine-grained-scaled A[M,K] . B[N,K]^T (see include/dg.h)."""
    _fp8(a, "a"); _fp8(b, "b"); _f32(sa, "sa"); _f32(sb, "sb")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b"); _shape(sa, (m, k // 128), "sa"); _shape(sb, ((n + 127) // 128, k // 128), "sb")
    _shape(c, (m, n), "c")
    if c.dtype != torch.bfloat16:
        raise TypeError("c must be bfloat16")
    _dev(a, sa, b, sb, c)
    _check(_lib.dg_gemm_fp8_nt(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(c), m, n, k, _stream(c)),
           "dg_gemm_fp8_nt")
    return c


def dg_gemm_fp8_nt_ue8m0(a, sa, b, sb, c):
    """dg_gemm_fp8_nt with power-of-two (UE8M0) scales applied by the
    block-scaled MFMA (see include/dg.h); sa, sb must be powers of two."""
    _fp8(a, "a"); _fp8(b, "b"); _f32(sa, "sa"); _f32(sb, "sb")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b"); _shape(sa, (m, k // 128), "sa"); _shape(sb, ((n + 127) // 128, k // 128), "sb")
    _shape(c, (m, n), "c")
    if c.dtype != torch.bfloat16:
        raise TypeError("c must be bfloat16")
    _dev(a, sa, b, sb, c)
    _check(_lib.dg_gemm_fp8_nt_ue8m0(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(c), m, n, k, _stream(c)),
           "dg_gemm_fp8_nt_ue8m0")
    return c


def dg_gemm_fp8_nt_ue8m0_packed(a, sa, b, sb, c):
    """dg_gemm_fp8_nt_ue8m0 with packed UE8M0 scales: int32 words holding the
    biased exponents of four consecutive K blocks, block 4w+i in byte i
    (sa [M, ceil(K/512)], sb [ceil(N/128), ceil(K/512)]; see include/dg.h)."""
    _fp8(a, "a"); _fp8(b, "b")
    for t, name in ((sa, "sa"), (sb, "sb")):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32 (packed UE8M0), got {t.dtype}")
    m, k = a.shape
    n = b.shape[0]
    kw = (k // 128 + 3) // 4
    _shape(b, (n, k), "b"); _shape(sa, (m, kw), "sa"); _shape(sb, ((n + 127) // 128, kw), "sb")
    _shape(c, (m, n), "c")
    if c.dtype != torch.bfloat16:
        raise TypeError("c must be bfloat16")
    _dev(a, sa, b, sb, c)
    _check(_lib.dg_gemm_fp8_nt_ue8m0_packed(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(c), m, n, k, _stream(c)),
           "dg_gemm_fp8_nt_ue8m0_packed")
    return c


def dg_gemm_bf16_nt(a, b, c):
    """C[M,N] bf16 = A[M,K] bf16 . B[N,K]^T bf16, fp32 accumulation (see include/dg.h)."""
    for t, name in ((a, "a"), (b, "b"), (c, "c")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b"); _shape(c, (m, n), "c")
    _dev(a, b, c)
    _check(_lib.dg_gemm_bf16_nt(_ptr(a), _ptr(b), _ptr(c), m, n, k, _stream(c)), "dg_gemm_bf16_nt")
    return c


def _scale_cols(sa, sb, k, packed):
    """Columns of the scale tensors: K/128 fp32 scales, or ceil(K/512) int32
    words of packed UE8M0 exponents."""
    if not packed:
        _f32(sa, "sa"); _f32(sb, "sb")
        return k // 128
    for t, name in ((sa, "sa"), (sb, "sb")):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32 (packed UE8M0), got {t.dtype}")
    return (k // 128 + 3) // 4


def dg_grouped_bf16_contiguous(a, b, c, m_indices):
    """Contiguous MoE layout in BF16: a [M_total,K], b [G,N,K], c [M_total,N]
    bf16, m_indices [M_total] int32 (see include/dg.h)."""
    for t, name in ((a, "a"), (b, "b"), (c, "c")):
        _bf16(t, name)
    m_total, k = a.shape
    g, n, _ = b.shape
    _shape(b, (g, n, k), "b"); _shape(c, (m_total, n), "c"); _shape(m_indices, (m_total,), "m_indices")
    if m_indices.dtype != torch.int32:
        raise TypeError("m_indices must be int32")
    _dev(a, b, c, m_indices)
    _check(_lib.dg_grouped_bf16_contiguous(_ptr(a), _ptr(b), _ptr(c), _ptr(m_indices), m_total, n, k, g, _stream(c)),
           "dg_grouped_bf16_contiguous")
    return c


def dg_grouped_bf16_masked(a, b, c, masked_m):
    """Masked MoE layout in BF16: a [G,M_max,K], b [G,N,K], c [G,M_max,N] bf16,
    masked_m [G] int32 (see include/dg.h)."""
    for t, name in ((a, "a"), (b, "b"), (c, "c")):
        _bf16(t, name)
    g, m_max, k = a.shape
    n = b.shape[1]
    _shape(b, (g, n, k), "b"); _shape(c, (g, m_max, n), "c"); _shape(masked_m, (g,), "masked_m")
    if masked_m.dtype != torch.int32:
        raise TypeError("masked_m must be int32")
    _dev(a, b, c, masked_m)
    _check(_lib.dg_grouped_bf16_masked(_ptr(a), _ptr(b), _ptr(c), _ptr(masked_m), g, m_max, n, k, _stream(c)),
           "dg_grouped_bf16_masked")
    return c


def dg_grouped_fp8_contiguous(a, sa, b, sb, c, m_indices):
    return _grouped_contiguous(_lib.dg_grouped_fp8_contiguous, "dg_grouped_fp8_contiguous", False,
                               a, sa, b, sb, c, m_indices)


def dg_grouped_fp8_contiguous_ue8m0_packed(a, sa, b, sb, c, m_indices):
    """dg_grouped_fp8_contiguous with packed UE8M0 scales (int32 words of four
    exponent bytes: sa [M_total, ceil(K/512)], sb [G, ceil(N/128), ceil(K/512)])."""
    return _grouped_contiguous(_lib.dg_grouped_fp8_contiguous_ue8m0_packed,
                               "dg_grouped_fp8_contiguous_ue8m0_packed", True, a, sa, b, sb, c, m_indices)


def _grouped_contiguous(fn, name, packed, a, sa, b, sb, c, m_indices):
    _fp8(a, "a"); _fp8(b, "b")
    m_total, k = a.shape
    g, n, _ = b.shape
    kc = _scale_cols(sa, sb, k, packed)
    _shape(b, (g, n, k), "b"); _shape(sa, (m_total, kc), "sa")
    _shape(sb, (g, (n + 127) // 128, kc), "sb"); _shape(c, (m_total, n), "c")
    _shape(m_indices, (m_total,), "m_indices")
    if m_indices.dtype != torch.int32:
        raise TypeError("m_indices must be int32")
    if c.dtype != torch.bfloat16:
        raise TypeError("c must be bfloat16")
    _dev(a, sa, b, sb, c, m_indices)
    _check(fn(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(c), _ptr(m_indices), m_total, n, k, g, _stream(c)), name)
    return c


def dg_grouped_fp8_contiguous_swiglu(a, sa, b, sb, q, s, m_indices):
    """Contiguous grouped GEMM with B [G,2I,K] (gate rows | up rows), fused
    with SwiGLU and the 1x128 re-quantise: q fp8 [M_total,I], s fp32
    [M_total,I/128] (see include/dg.h)."""
    _fp8(a, "a"); _fp8(b, "b"); _f32(sa, "sa"); _f32(sb, "sb"); _fp8(q, "q"); _f32(s, "s")
    m_total, k = a.shape
    g, n, _ = b.shape
    if n % 256:
        raise ValueError(f"b must stack gate and up projections of a width that is a multiple of 128 (N={n})")
    i = n // 2
    _shape(b, (g, n, k), "b"); _shape(sa, (m_total, k // 128), "sa")
    _shape(sb, (g, n // 128, k // 128), "sb"); _shape(q, (m_total, i), "q"); _shape(s, (m_total, i // 128), "s")
    _shape(m_indices, (m_total,), "m_indices")
    if m_indices.dtype != torch.int32:
        raise TypeError("m_indices must be int32")
    _dev(a, sa, b, sb, q, s, m_indices)
    _check(_lib.dg_grouped_fp8_contiguous_swiglu(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(q), _ptr(s),
                                                 _ptr(m_indices), m_total, n, k, g, _stream(q)),
           "dg_grouped_fp8_contiguous_swiglu")
    return q, s


def dg_grouped_fp8_masked(a, sa, b, sb, c, masked_m):
    return _grouped_masked(_lib.dg_grouped_fp8_masked, "dg_grouped_fp8_masked", a, sa, b, sb, c, masked_m)


def dg_grouped_fp8_masked_ue8m0_packed(a, sa, b, sb, c, masked_m):
    """dg_grouped_fp8_masked with packed UE8M0 scales (int32 words of four
    exponent bytes: sa [G, M_max, ceil(K/512)], sb [G, ceil(N/128), ceil(K/512)])."""
    return _grouped_masked(_lib.dg_grouped_fp8_masked_ue8m0_packed, "dg_grouped_fp8_masked_ue8m0_packed",
                           a, sa, b, sb, c, masked_m, packed=True)


def dg_grouped_fp8_masked_noalloc(a, sa, b, sb, c, masked_m):
    """dg_grouped_fp8_masked without any allocation (split-K partials in the
    library's fixed 64 MB scratch; usable under graph capture).  Calls that
    overlap on one GPU share the scratch and race."""
    return _grouped_masked(_lib.dg_grouped_fp8_masked_noalloc, "dg_grouped_fp8_masked_noalloc",
                           a, sa, b, sb, c, masked_m)


def _grouped_masked(fn, name, a, sa, b, sb, c, masked_m, packed=False):
    _fp8(a, "a"); _fp8(b, "b")
    g, m_max, k = a.shape
    n = b.shape[1]
    kc = _scale_cols(sa, sb, k, packed)
    _shape(b, (g, n, k), "b"); _shape(sa, (g, m_max, kc), "sa")
    _shape(sb, (g, (n + 127) // 128, kc), "sb"); _shape(c, (g, m_max, n), "c")
    _shape(masked_m, (g,), "masked_m")
    if masked_m.dtype != torch.int32:
        raise TypeError("masked_m must be int32")
    if c.dtype != torch.bfloat16:
        raise TypeError("c must be bfloat16")
    _dev(a, sa, b, sb, c, masked_m)
    _check(fn(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(c), _ptr(masked_m), g, m_max, n, k, _stream(c)), name)
    return c


def dg_wgrad_fp8_nt(a, sa, b, sb, d):
    _fp8(a, "a"); _fp8(b, "b"); _f32(sa, "sa"); _f32(sb, "sb")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b"); _shape(sa, (m, k // 128), "sa"); _shape(sb, (n, k // 128), "sb")
    _shape(d, (m, n), "d"); _f32(d, "d")
    _dev(a, sa, b, sb, d)
    _check(_lib.dg_wgrad_fp8_nt(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), m, n, k, _stream(d)),
           "dg_wgrad_fp8_nt")
    return d


def dg_k_grouped_wgrad_fp8_nt(a, sa, b, sb, d, ks):
    """ks: per-group token counts (host list/tuple of ints, multiples of 128)."""
    _fp8(a, "a"); _fp8(b, "b"); _f32(sa, "sa"); _f32(sb, "sb")
    ks = [int(x) for x in ks]
    g = len(ks)
    m, t = a.shape
    n = b.shape[0]
    if sum(ks) != t:
        raise ValueError(f"sum(ks)={sum(ks)} does not match the token dimension {t}")
    _shape(b, (n, t), "b"); _shape(sa, (m, t // 128), "sa"); _shape(sb, (n, t // 128), "sb")
    _shape(d, (g, m, n), "d"); _f32(d, "d")
    _dev(a, sa, b, sb, d)
    ks_arr = (ctypes.c_int32 * g)(*ks)
    _check(_lib.dg_k_grouped_wgrad_fp8_nt(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), ks_arr, g, m, n,
                                          _stream(d)), "dg_k_grouped_wgrad_fp8_nt")
    return d


def dg_quantize_fp8_1x128(x, q, s):
    """x fp32 [M,K] -> q fp8 [M,K], s fp32 [M,K/128] (see include/dg.h)."""
    _f32(x, "x"); _fp8(q, "q"); _f32(s, "s")
    _dev(x, q, s)
    m, k = x.shape
    _shape(q, (m, k), "q"); _shape(s, (m, k // 128), "s")
    _check(_lib.dg_quantize_fp8_1x128(_ptr(x), _ptr(q), _ptr(s), m, k, _stream(x)), "dg_quantize_fp8_1x128")
    return q, s


def dg_quantize_fp8_128x128(x, q, s):
    """x fp32 [N,K] -> q fp8 [N,K], s fp32 [ceil(N/128),K/128] (see include/dg.h)."""
    _f32(x, "x"); _fp8(q, "q"); _f32(s, "s")
    _dev(x, q, s)
    n, k = x.shape
    _shape(q, (n, k), "q"); _shape(s, ((n + 127) // 128, k // 128), "s")
    _check(_lib.dg_quantize_fp8_128x128(_ptr(x), _ptr(q), _ptr(s), n, k, _stream(x)), "dg_quantize_fp8_128x128")
    return q, s


def _i32w(t, name):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32 (packed UE8M0), got {t.dtype}")


def dg_quantize_fp8_1x128_ue8m0(x, q, s):
    """x fp32 [M,K] -> q fp8 [M,K], s int32 [M,ceil(K/512)]: power-of-two
    scales, packed UE8M0 (see include/dg.h)."""
    _f32(x, "x"); _fp8(q, "q"); _i32w(s, "s")
    _dev(x, q, s)
    m, k = x.shape
    _shape(q, (m, k), "q"); _shape(s, (m, (k // 128 + 3) // 4), "s")
    _check(_lib.dg_quantize_fp8_1x128_ue8m0(_ptr(x), _ptr(q), _ptr(s), m, k, _stream(x)),
           "dg_quantize_fp8_1x128_ue8m0")
    return q, s


def dg_quantize_fp8_128x128_ue8m0(x, q, s):
    """x fp32 [N,K] -> q fp8 [N,K], s int32 [ceil(N/128),ceil(K/512)]: power-of-two
    scales, packed UE8M0 (see include/dg.h)."""
    _f32(x, "x"); _fp8(q, "q"); _i32w(s, "s")
    _dev(x, q, s)
    n, k = x.shape
    _shape(q, (n, k), "q"); _shape(s, ((n + 127) // 128, (k // 128 + 3) // 4), "s")
    _check(_lib.dg_quantize_fp8_128x128_ue8m0(_ptr(x), _ptr(q), _ptr(s), n, k, _stream(x)),
           "dg_quantize_fp8_128x128_ue8m0")
    return q, s


def dg_quantize_fp8_1x128_transposed(x, q, s):
    """x fp32 [T,F] -> q fp8 [F,T], s fp32 [F,T/128] (see include/dg.h)."""
    _f32(x, "x"); _fp8(q, "q"); _f32(s, "s")
    _dev(x, q, s)
    t, f = x.shape
    _shape(q, (f, t), "q"); _shape(s, (f, t // 128), "s")
    _check(_lib.dg_quantize_fp8_1x128_transposed(_ptr(x), _ptr(q), _ptr(s), t, f, _stream(x)),
           "dg_quantize_fp8_1x128_transposed")
    return q, s


def _even_width(c):
    """(M, 2I) of the first GEMM's output c: the gate and up halves need an
    even width (an odd one would walk the rows with the wrong stride)."""
    if c.dim() != 2 or c.shape[1] % 2:
        raise ValueError(f"c must be [M, 2I] with an even width, got {tuple(c.shape)}")
    return c.shape


def dg_swiglu_quantize_fp8_1x128(c, q, s):
    """c bf16 [M,2I] (gate | up) -> q fp8 [M,I], s fp32 [M,I/128]: SwiGLU then
    the 1x128 quantise (see include/dg.h)."""
    _bf16(c, "c"); _fp8(q, "q"); _f32(s, "s")
    m, i2 = _even_width(c)
    _dev(c, q, s)
    i = i2 // 2
    _shape(q, (m, i), "q"); _shape(s, (m, i // 128), "s")
    _check(_lib.dg_swiglu_quantize_fp8_1x128(_ptr(c), _ptr(q), _ptr(s), m, i, _stream(c)),
           "dg_swiglu_quantize_fp8_1x128")
    return q, s


# -------------------------------------- linear layer with its epilogue ---

_ACTIVATION = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_TYPE = {torch.bfloat16: 0, torch.float32: 1}


def _activation(name):
    a = _ACTIVATION.get(name)
    if a is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATION)}, got {name!r}")
    return a


def _ld(t, dev, name):
    """Row stride of a 2-D tensor with contiguous rows on GPU `dev`."""
    if t.get_device() != dev:  # -1 on the host
        raise ValueError("all tensors must be on the same GPU")
    ld, one = t.stride()
    rows, cols = t.shape
    if (one != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name} must have contiguous, non-overlapping rows")
    return ld if rows > 1 else cols  # one row: its stride may be anything (x[:, -1] of one sequence)


def _epilogue(out, bias, activation, residual, pre, m, n, dev):
    e = _Epilogue()
    e.activation = _activation(activation)
    if bias is not None:
        if bias.dtype not in _TYPE:
            raise TypeError(f"bias must be bfloat16 or float32, got {bias.dtype}")
        if bias.shape != (n,) or (n > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be contiguous with shape {(n,)}, got {tuple(bias.shape)}")
        if bias.get_device() != dev:
            raise ValueError("all tensors must be on the same GPU")
        e.bias, e.bias_type = _ptr(bias), _TYPE[bias.dtype]
    if residual is not None:
        _bf16(residual, "residual"); _shape(residual, (m, n), "residual")
        e.residual, e.ld_residual = _ptr(residual), _ld(residual, dev, "residual")
    if pre is not None:
        _bf16(pre, "pre"); _shape(pre, (m, n), "pre")
        e.pre, e.ld_pre = _ptr(pre), _ld(pre, dev, "pre")
    return e


def _linear_out(out, m, n, dev):
    if out.dtype not in _TYPE:
        raise TypeError(f"out must be bfloat16 or float32, got {out.dtype}")
    _shape(out, (m, n), "out")
    return _ld(out, dev, "out")


def _gpu(t):
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    return t.get_device()


def gemm_bf16_nt_epilogue(a, b, out, bias=None, activation="none", residual=None, pre=None):
    """out[M,N] = activation(a[M,K] . b[N,K]^T + bias) + residual in BF16 (see
    dg_gemm_bf16_nt_epilogue in include/dg.h).  out bf16 or fp32; bias [N] bf16
    or fp32; residual [M,N] bf16 (may be out); pre [M,N] bf16 receives the
    pre-activation for the backward pass.  Rows may be strided."""
    _bf16(a, "a"); _bf16(b, "b")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b")
    dev = _gpu(a)
    ldc = _linear_out(out, m, n, dev)
    e = _epilogue(out, bias, activation, residual, pre, m, n, dev)
    _check(_lib.dg_gemm_bf16_nt_epilogue(_ptr(a), _ld(a, dev, "a"), _ptr(b), _ld(b, dev, "b"), _ptr(out), ldc,
                                         _TYPE[out.dtype], ctypes.addressof(e), m, n, k, _stream(a)),
           "dg_gemm_bf16_nt_epilogue")
    return out


def gemm_fp8_nt_epilogue(lhs, rhs, out, bias=None, activation="none", residual=None, pre=None):
    """gemm_bf16_nt_epilogue on FP8 operands with their scales: lhs = (fp8
    [M,K], fp32 [M,K/128]), rhs = (fp8 [N,K], fp32 [ceil(N/128),K/128])."""
    (a, sa), (b, sb) = lhs, rhs
    _fp8(a, "a"); _fp8(b, "b"); _f32(sa, "sa"); _f32(sb, "sb")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b"); _shape(sa, (m, k // 128), "sa"); _shape(sb, ((n + 127) // 128, k // 128), "sb")
    _dev(a, sa, b, sb)
    dev = a.get_device()
    ldc = _linear_out(out, m, n, dev)
    e = _epilogue(out, bias, activation, residual, pre, m, n, dev)
    _check(_lib.dg_gemm_fp8_nt_epilogue(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), ldc, _TYPE[out.dtype],
                                        ctypes.addressof(e), m, n, k, _stream(a)),
           "dg_gemm_fp8_nt_epilogue")
    return out


def gemm_bf16_nt_epilogue_backward_workspace(m, n):
    """Bytes of workspace that gemm_bf16_nt_epilogue_backward needs for dout [m,n]."""
    need = _i64()
    _check(_lib.dg_gemm_bf16_nt_epilogue_backward_workspace(m, n, ctypes.byref(need)),
           "dg_gemm_bf16_nt_epilogue_backward_workspace")
    return need.value


def gemm_bf16_nt_epilogue_backward(dout, a, b, pre=None, activation="none", da=None, db=None, dbias=None,
                                   workspace=None):
    """Gradients of gemm_bf16_nt_epilogue from dout bf16 [M,N] and the stored
    pre-activation (see include/dg.h): writes those of da bf16 [M,K], db bf16
    [N,K] and dbias fp32 [N] that are given and returns the three.  The
    residual's gradient is dout."""
    _bf16(dout, "dout"); _bf16(a, "a"); _bf16(b, "b")
    m, k = a.shape
    n = b.shape[0]
    _shape(b, (n, k), "b"); _shape(dout, (m, n), "dout")
    dev = _gpu(dout)
    act = _activation(activation)
    if act and pre is None:
        raise ValueError(f"activation {activation!r} needs the stored pre-activation")
    pp, ldp = None, 0
    if act:
        _bf16(pre, "pre"); _shape(pre, (m, n), "pre")
        pp, ldp = _ptr(pre), _ld(pre, dev, "pre")
    pa = pb = pbias = None
    lda = ldb = 0
    if da is not None:
        _bf16(da, "da"); _shape(da, (m, k), "da")
        pa, lda = _ptr(da), _ld(da, dev, "da")
    if db is not None:
        _bf16(db, "db"); _shape(db, (n, k), "db")
        pb, ldb = _ptr(db), _ld(db, dev, "db")
    if dbias is not None:
        _f32(dbias, "dbias"); _shape(dbias, (n,), "dbias")
        if dbias.get_device() != dev or not dbias.is_contiguous():
            raise ValueError("dbias must be contiguous, on the same GPU")
        pbias = _ptr(dbias)
    need = gemm_bf16_nt_epilogue_backward_workspace(m, n)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dout.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be contiguous, on the same GPU, with at least {need} bytes")
    _check(_lib.dg_gemm_bf16_nt_epilogue_backward(
        _ptr(dout), _ld(dout, dev, "dout"), _ptr(a), _ld(a, dev, "a"), _ptr(b), _ld(b, dev, "b"), pp, ldp, act,
        pa, lda, pb, ldb, pbias, _ptr(workspace), m, n, k, _stream(dout)), "dg_gemm_bf16_nt_epilogue_backward")
    return da, db, dbias


# ------------------------------------- a whole MoE layer for a few tokens ---

_SCORING = {"softmax": 0, "sigmoid": 1}


def _moe_few_tokens(name, fp8, x, w13, w2, out, ids, weights, logits, scoring, renormalize, scale, residual,
                    workspace):
    _bf16(x, "x"); _bf16(out, "out"); _f32(weights, "weights")
    if fp8:
        (w13, s13), (w2, s2) = w13, w2
        _fp8(w13, "w13"); _fp8(w2, "w2"); _f32(s13, "s13"); _f32(s2, "s2")
    else:
        _bf16(w13, "w13"); _bf16(w2, "w2")
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    t, h = x.shape
    e, n, _ = w13.shape
    if n % 256:
        raise ValueError(f"w13 must stack gate and up projections of a width that is a multiple of 128 (2I={n})")
    i = n // 2
    k = ids.shape[-1]
    _shape(w13, (e, n, h), "w13"); _shape(w2, (e, h, i), "w2"); _shape(out, (t, h), "out")
    _shape(ids, (t, k), "ids"); _shape(weights, (t, k), "weights")
    tensors = [x, w13, w2, out, ids, weights]
    if fp8:
        _shape(s13, (e, n // 128, h // 128), "s13"); _shape(s2, (e, h // 128, i // 128), "s2")
        tensors += [s13, s2]
    if logits is not None:
        _f32(logits, "logits"); _shape(logits, (t, e), "logits")
        tensors.append(logits)
    if residual is not None:
        _bf16(residual, "residual"); _shape(residual, (t, h), "residual")
        tensors.append(residual)
    if workspace is None:
        workspace = torch.empty(t * k * i, dtype=torch.bfloat16, device=x.device)
    elif workspace.numel() * workspace.element_size() < 2 * t * k * i:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, {2 * t * k * i} needed")
    tensors.append(workspace)
    _dev(*tensors)
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    lg = None if logits is None else _ptr(logits)
    rs = None if residual is None else _ptr(residual)
    tail = (rs, _ptr(out), _ptr(workspace), t, h, i, e, k, _SCORING[scoring], 1 if renormalize else 0, scale,
            _stream(x))
    if fp8:
        st = _lib.dg_moe_few_tokens_fp8(_ptr(x), lg, _ptr(ids), _ptr(weights), _ptr(w13), _ptr(s13), _ptr(w2),
                                        _ptr(s2), *tail)
    else:
        st = _lib.dg_moe_few_tokens_bf16(_ptr(x), lg, _ptr(ids), _ptr(weights), _ptr(w13), _ptr(w2), *tail)
    _check(st, name)
    return out


def moe_few_tokens_fp8(x, w13, w2, out, ids, weights, logits=None, scoring="softmax", renormalize=True, scale=1.0,
                       residual=None, workspace=None):
    """A whole MoE layer for 1..64 tokens on FP8 weights (see include/dg.h):
    x bf16 [T,H], w13 = (fp8 [E,2I,H], fp32 [E,2I/128,H/128]) with the gate
    rows first, w2 = (fp8 [E,H,I], fp32 [E,H/128,I/128]), out bf16 [T,H].
    With logits fp32 [T,E] the call routes and writes ids int32 [T,k] and
    weights fp32 [T,k]; without, it reads them."""
    return _moe_few_tokens("dg_moe_few_tokens_fp8", True, x, w13, w2, out, ids, weights, logits, scoring,
                           renormalize, scale, residual, workspace)


def moe_few_tokens_bf16(x, w13, w2, out, ids, weights, logits=None, scoring="softmax", renormalize=True, scale=1.0,
                        residual=None, workspace=None):
    """moe_few_tokens_fp8 on BF16 weights w13 [E,2I,H] and w2 [E,H,I]."""
    return _moe_few_tokens("dg_moe_few_tokens_bf16", False, x, w13, w2, out, ids, weights, logits, scoring,
                           renormalize, scale, residual, workspace)


# ------------------------- norm with the residual's addition, INT8 layer ---
# Small calls are bound by what happens before the launch, so each tensor is
# looked at once, natively (csrc/dg_tensors.cpp).  The functions in Python that
# have a native counterpart (_matrix_of for _matrix, ...) answer where that finds
# anything unexpected: they work out the reason and raise.  Without the native
# module they do all of it.

_BF16, _F32, _I32, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
_norm_fields = struct.Struct("PqPqPifPqP").pack   # dg_norm
_epilogue_fields = struct.Struct("PiiPqPq").pack  # dg_epilogue


def _device_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


_stream_of = _raw_stream or _device_stream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _refuse(t, dtype, shape, dev, name):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same GPU as the call's first tensor")
    raise ValueError(f"{name} must be contiguous (a matrix whose stride the call takes: contiguous rows that do not "
                     f"overlap), got strides {t.stride()}")


def _fitting(t, dtype, shape, dev, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t)}")
    return (t.layout is torch.strided and t.dtype is dtype and t.shape == tuple(shape) and t.is_cuda
            and t.get_device() == dev)


def _whole_of(t, dtype, shape, dev, name):
    """Address of a contiguous tensor of the given type and shape on GPU `dev`."""
    if not _fitting(t, dtype, shape, dev, name) or not t.is_contiguous():
        _refuse(t, dtype, shape, dev, name)
    return t.data_ptr()


def _rows_of(t, dtype, shape, dev, name):
    """Address and row stride of a matrix with contiguous rows (one row: its stride may be anything)."""
    if not _fitting(t, dtype, shape, dev, name) or t.dim() != 2:
        _refuse(t, dtype, shape, dev, name)
    (m, cols), (ld, one) = shape, t.stride()
    if (one != 1 and cols > 1) or (ld < cols and m > 1):
        _refuse(t, dtype, shape, dev, name)
    return t.data_ptr(), ld if m > 1 else cols


if _tensors is not None:
    _tensors.refuse_with(_refuse)
    _whole, _rows = _tensors.whole, _tensors.rows
else:
    _whole, _rows = _whole_of, _rows_of


def _bytes8_of(t, shape, dev, name):
    """Pointer of a contiguous tensor of FP8 values or their bytes."""
    _fp8(t, name)
    return _whole(t, t.dtype, shape, dev, name)


def _vector_of(t, n, dev, name):
    """Pointer and type of a contiguous vector in bf16 or fp32."""
    kind = _TYPE.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return _whole(t, t.dtype, (n,), dev, name), kind


def _matrix_of(t, name, current):
    """Shape and GPU of a call's first tensor."""
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(t.shape)}")
    dev = t.get_device()
    if dev != current():  # (the default stream is the current GPU's)
        raise ValueError(f"{name} is on GPU {dev}, which is not the current one: call under torch.cuda.device({dev})")
    return t.shape, dev


def _room(workspace, need, dev, like):
    """A workspace of at least `need` bytes, made if there is none, and its pointer.  The caller holds it until the
    library has launched: freed before, another thread's tensor could take its place."""
    if not need:
        return None, None
    if workspace is None:
        workspace = like.new_empty(need, dtype=torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be contiguous, on the same GPU, with at least {need} bytes")
    return workspace, workspace.data_ptr()


def _norm_of(x, shape, weight, eps, residual, sum_out, rstd, dev):
    """The call's dg_norm, as bytes."""
    xp, ldx = _rows(x, _BF16, shape, dev, "x")
    wp = rp = sp = dp = wt = ldr = lds = 0
    if weight is not None:
        wp, wt = _vector_of(weight, shape[1], dev, "weight")
    if residual is not None:
        rp, ldr = _rows(residual, _BF16, shape, dev, "residual")
    if sum_out is not None:
        sp, lds = _rows(sum_out, _BF16, shape, dev, "sum_out")
    if rstd is not None:
        dp = _whole(rstd, _F32, shape[:1], dev, "rstd")
    return _norm_fields(xp, ldx, rp, ldr, wp, wt, eps, sp, lds, dp)


def _layout_of(a, dtype, cols, dev, name):
    """Pointer and row count of a grouped layout's rows [M,cols] or [E,M_max,cols]
    (dtype None: FP8 values or their bytes)."""
    if dtype is None:
        _fp8(a, name)
        dtype = a.dtype
    shape = a.shape
    n = len(shape)
    if n not in (2, 3) or shape[-1] != cols:
        raise ValueError(f"{name} must be [M,{cols}] or [E,M_max,{cols}], got {tuple(shape)}")
    return _whole(a, dtype, shape, dev, name), shape[0] if n == 2 else shape[0] * shape[1]


def _slots_of(rows, t, dev):
    """Pointer and width of the rows int32 [T,k] of the tokens' slots."""
    shape = rows.shape
    if len(shape) != 2 or shape[0] != t:
        raise ValueError(f"rows must be [{t},k], got {tuple(shape)}")
    return _whole(rows, _I32, shape, dev, "rows"), shape[1]


if _tensors is not None:
    _tensors.otherwise(_matrix_of, _vector_of, _bytes8_of, _layout_of, _slots_of, _norm_of)
    _matrix, _vector, _bytes8 = _tensors.matrix, _tensors.vector, _tensors.bytes8
    _layout, _slots, _norm = _tensors.layout, _tensors.slots, _tensors.norm
else:
    _matrix, _vector, _bytes8, _layout, _slots, _norm = _matrix_of, _vector_of, _bytes8_of, _layout_of, _slots_of, _norm_of


def rmsnorm_bf16(x, weight, out, eps=1e-6, residual=None, sum_out=None, rstd=None):
    """out bf16 [T,H] = z / sqrt(mean(z^2) + eps) * weight with z = x + residual
    (see dg_rmsnorm_bf16 in include/dg.h).  weight [H] bf16, fp32 or None;
    sum_out bf16 [T,H] receives z (may be x or residual), rstd fp32 [T] the
    factor for the backward pass.  Rows may be strided."""
    shape, dev = _matrix(x, "x", _current_device)
    p = _norm(x, shape, weight, eps, residual, sum_out, rstd, dev)
    op, ldo = _rows(out, _BF16, shape, dev, "out")
    st = _lib.dg_rmsnorm_bf16(p, op, ldo, *shape, _stream_of(dev))
    if st:
        raise DGError(st, "dg_rmsnorm_bf16")
    return out


def rmsnorm_quantize_fp8_1x128(x, weight, q, s, eps=1e-6, residual=None, sum_out=None, rstd=None):
    """rmsnorm_bf16 with its fp32 result quantised: q fp8 [T,H], s fp32
    [T,H/128], or int32 [T,ceil(H/512)] for packed UE8M0 scales."""
    shape, dev = _matrix(x, "x", _current_device)
    t, h = shape
    p = _norm(x, shape, weight, eps, residual, sum_out, rstd, dev)
    qp = _bytes8(q, shape, dev, "q")
    if s.dtype is _I32:
        fn, name, sp = _lib.dg_rmsnorm_quantize_fp8_1x128_ue8m0, "dg_rmsnorm_quantize_fp8_1x128_ue8m0", \
            _whole(s, _I32, (t, (h + 511) // 512), dev, "s")
    else:
        fn, name, sp = _lib.dg_rmsnorm_quantize_fp8_1x128, "dg_rmsnorm_quantize_fp8_1x128", \
            _whole(s, _F32, (t, h // 128), dev, "s")
    st = fn(p, qp, sp, t, h, _stream_of(dev))
    if st:
        raise DGError(st, name)
    return q, s


def rmsnorm_quantize_int8(x, weight, q, s, eps=1e-6, residual=None, sum_out=None, rstd=None):
    """rmsnorm_bf16 with its fp32 result quantised: q int8 [T,H], s fp32 [T]."""
    shape, dev = _matrix(x, "x", _current_device)
    p = _norm(x, shape, weight, eps, residual, sum_out, rstd, dev)
    st = _lib.dg_rmsnorm_quantize_int8(p, _whole(q, _I8, shape, dev, "q"), _whole(s, _F32, shape[:1], dev, "s"), *shape,
                                       _stream_of(dev))
    if st:
        raise DGError(st, "dg_rmsnorm_quantize_int8")
    return q, s


@functools.lru_cache(maxsize=256)
def rmsnorm_bf16_backward_workspace(t, h):
    """Bytes of workspace that rmsnorm_bf16_backward needs for dweight."""
    need = _i64()
    _check(_lib.dg_rmsnorm_bf16_backward_workspace(t, h, ctypes.byref(need)), "dg_rmsnorm_bf16_backward_workspace")
    return need.value


def rmsnorm_bf16_backward(dout, z, weight, rstd, dx=None, dweight=None, dsum=None, workspace=None):
    """Gradients of the norm from dout bf16 [T,H], the stored sum z bf16 [T,H]
    (or x) and rstd fp32 [T] (see include/dg.h): writes those of dx bf16 [T,H]
    (the gradient of x and of residual; dsum bf16 [T,H], the gradient that
    reaches sum_out from elsewhere, is added) and dweight fp32 [H] that are
    given and returns both."""
    shape, dev = _matrix(dout, "dout", _current_device)
    t, h = shape
    op, ldo = _rows(dout, _BF16, shape, dev, "dout")
    zp, ldz = _rows(z, _BF16, shape, dev, "z")
    wp, wt = (None, 0) if weight is None else _vector(weight, h, dev, "weight")
    dsp = dxp = dwp = wsp = None
    ldds = lddx = 0
    if dx is not None:
        dxp, lddx = _rows(dx, _BF16, shape, dev, "dx")
        if dsum is not None:
            dsp, ldds = _rows(dsum, _BF16, shape, dev, "dsum")
    if dweight is not None:
        dwp = _whole(dweight, _F32, (h,), dev, "dweight")
        workspace, wsp = _room(workspace, rmsnorm_bf16_backward_workspace(t, h), dev, dout)
    st = _lib.dg_rmsnorm_bf16_backward(op, ldo, zp, ldz, wp, wt, _whole(rstd, _F32, (t,), dev, "rstd"), dsp, ldds, dxp,
                                       lddx, dwp, wsp, t, h, _stream_of(dev))
    if st:
        raise DGError(st, "dg_rmsnorm_bf16_backward")
    return dx, dweight


def gemm_int8_nt_epilogue(lhs, rhs, out, bias=None, activation="none", residual=None, pre=None):
    """gemm_bf16_nt_epilogue on INT8 operands with a scale per row: lhs = (int8
    [M,K], fp32 [M]), rhs = (int8 [N,K], fp32 [N]) (see
    dg_gemm_int8_nt_epilogue in include/dg.h)."""
    (a, sa), (b, sb) = lhs, rhs
    (m, k), dev = _matrix(a, "a", _current_device)
    n = b.shape[0]
    ap, lda = _rows(a, _I8, (m, k), dev, "a")
    bp, ldb = _rows(b, _I8, (n, k), dev, "b")
    kind = _TYPE.get(out.dtype)
    if kind is None:
        raise TypeError(f"out must be bfloat16 or float32, got {out.dtype}")
    cp, ldc = _rows(out, out.dtype, (m, n), dev, "out")
    bip = bit = rp = ldr = pp = ldp = 0
    if bias is not None:
        bip, bit = _vector(bias, n, dev, "bias")
    if residual is not None:
        rp, ldr = _rows(residual, _BF16, (m, n), dev, "residual")
    if pre is not None:
        pp, ldp = _rows(pre, _BF16, (m, n), dev, "pre")
    st = _lib.dg_gemm_int8_nt_epilogue(ap, lda, _whole(sa, _F32, (m,), dev, "sa"), bp, ldb,
                                       _whole(sb, _F32, (n,), dev, "sb"), cp, ldc, kind,
                                       _epilogue_fields(bip, bit, _activation(activation), rp, ldr, pp, ldp), m, n, k,
                                       _stream_of(dev))
    if st:
        raise DGError(st, "dg_gemm_int8_nt_epilogue")
    return out


def dg_quantize_int8_rows(x, q, s):
    """x bf16 or fp32 [M,K] -> q int8 [M,K], s fp32 [M]: a scale per row (see
    include/dg.h).  x's rows may be strided."""
    shape, dev = _matrix(x, "x", _current_device)
    kind = _TYPE.get(x.dtype)
    if kind is None:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    xp, ldx = _rows(x, x.dtype, shape, dev, "x")
    st = _lib.dg_quantize_int8_rows(xp, ldx, kind, _whole(q, _I8, shape, dev, "q"),
                                    _whole(s, _F32, shape[:1], dev, "s"), *shape, _stream_of(dev))
    if st:
        raise DGError(st, "dg_quantize_int8_rows")
    return q, s


# ------------------------------------- tokens sorted by expert and back ---

@functools.lru_cache(maxsize=256)
def moe_sort_workspace(tokens, top_k, num_experts):
    """Bytes of workspace that moe_sort_contiguous and moe_sort_masked need."""
    need = _i64()
    _check(_lib.dg_moe_sort_workspace(tokens, top_k, num_experts, ctypes.byref(need)), "dg_moe_sort_workspace")
    return need.value


def moe_sort_rows(tokens, top_k, num_experts):
    """Rows of the contiguous layout that hold any routing (M_total)."""
    slots = tokens * top_k
    return max(128, (slots + min(num_experts, slots) * 127) // 128 * 128)


def moe_sort_contiguous(ids, num_experts, m_indices, rows, counts=None, workspace=None):
    """Rows of the contiguous layout for the tokens' experts ids int32 [T,k] (see
    dg_moe_sort_contiguous in include/dg.h): writes m_indices int32 [M_total]
    (moe_sort_rows gives an M_total for any routing), rows int32 [T,k] and, if
    given, counts int32 [E]; returns m_indices and rows."""
    shape, dev = _matrix(ids, "ids", _current_device)
    t, k = shape
    m = m_indices.shape[0]
    workspace, wsp = _room(workspace, moe_sort_workspace(t, k, num_experts), dev, ids)
    st = _lib.dg_moe_sort_contiguous(
        _whole(ids, _I32, shape, dev, "ids"), _whole(m_indices, _I32, (m,), dev, "m_indices"),
        _whole(rows, _I32, shape, dev, "rows"),
        None if counts is None else _whole(counts, _I32, (num_experts,), dev, "counts"), wsp, t, k, num_experts, m,
        _stream_of(dev))
    if st:
        raise DGError(st, "dg_moe_sort_contiguous")
    return m_indices, rows


def moe_sort_masked(ids, m_max, masked_m, rows, workspace=None):
    """Rows of the masked layout [E,M_max,..] for the tokens' experts ids int32
    [T,k]: writes masked_m int32 [E] and rows int32 [T,k] and returns both."""
    shape, dev = _matrix(ids, "ids", _current_device)
    t, k = shape
    e = masked_m.shape[0]
    workspace, wsp = _room(workspace, moe_sort_workspace(t, k, e), dev, ids)
    st = _lib.dg_moe_sort_masked(
        _whole(ids, _I32, shape, dev, "ids"), _whole(masked_m, _I32, (e,), dev, "masked_m"),
        _whole(rows, _I32, shape, dev, "rows"), wsp, t, k, e, m_max, _stream_of(dev))
    if st:
        raise DGError(st, "dg_moe_sort_masked")
    return masked_m, rows


def _optional(t, dtype, shape, dev, name):
    return None if t is None else _whole(t, dtype, shape, dev, name)


def moe_dispatch_bf16(x, rows, a, m_indices=None):
    """a[rows[t,j]] = x[t] for bf16 x [T,H] (see dg_moe_dispatch_bf16 in
    include/dg.h); a bf16 [M,H] or [E,M_max,H].  With m_indices (contiguous
    layout) the padding rows of the segments become zeros."""
    shape, dev = _matrix(x, "x", _current_device)
    t, h = shape
    xp, ldx = _rows(x, _BF16, shape, dev, "x")
    ap, m = _layout(a, _BF16, h, dev, "a")
    rp, k = _slots(rows, t, dev)
    st = _lib.dg_moe_dispatch_bf16(xp, ldx, rp, _optional(m_indices, _I32, (m,), dev, "m_indices"), ap, t, k, h, m,
                                   _stream_of(dev))
    if st:
        raise DGError(st, "dg_moe_dispatch_bf16")
    return a


def moe_dispatch_fp8(x, rows, a, m_indices=None):
    """moe_dispatch_bf16 for FP8 rows with their scales: x = (fp8 [T,H], fp32
    [T,H/128] or int32 [T,ceil(H/512)]), a = (fp8 [M,H] or [E,M_max,H], scales
    of the same)."""
    (q, s), (qa, sa) = x, a
    shape, dev = _matrix(q, "x", _current_device)
    t, h = shape
    qp = _bytes8(q, shape, dev, "x")
    ap, m = _layout(qa, None, h, dev, "a")
    kind = s.dtype
    if kind is _I32:
        fn, words = _lib.dg_moe_dispatch_fp8_ue8m0, (h + 511) // 512
    else:
        fn, words, kind = _lib.dg_moe_dispatch_fp8, h // 128, _F32
    sp = _whole(s, kind, (t, words), dev, "x's scales")
    sap, ms = _layout(sa, kind, words, dev, "a's scales")
    if ms != m:
        raise ValueError(f"a has {m} rows and its scales {ms}")
    rp, k = _slots(rows, t, dev)
    st = fn(qp, sp, rp, _optional(m_indices, _I32, (m,), dev, "m_indices"), ap, sap, t, k, h, m, _stream_of(dev))
    if st:
        raise DGError(st, "dg_moe_dispatch_fp8")
    return a


def moe_combine_bf16(o, rows, out, weights=None, residual=None):
    """out[t] = residual[t] + sum_j weights[t,j] o[rows[t,j]] (see
    dg_moe_combine_bf16 in include/dg.h): o bf16 [M,H] or [E,M_max,H], weights
    fp32 [T,k] or None (ones), residual bf16 [T,H] (may be out)."""
    shape, dev = _matrix(out, "out", _current_device)
    t, h = shape
    yp, ldy = _rows(out, _BF16, shape, dev, "out")
    op, m = _layout(o, _BF16, h, dev, "o")
    rp, k = _slots(rows, t, dev)
    res, ldr = (None, 0) if residual is None else _rows(residual, _BF16, shape, dev, "residual")
    st = _lib.dg_moe_combine_bf16(op, rp, _optional(weights, _F32, (t, k), dev, "weights"), res, ldr, yp, ldy, t, k, h, m,
                                  _stream_of(dev))
    if st:
        raise DGError(st, "dg_moe_combine_bf16")
    return out


def moe_dispatch_bf16_backward(da, rows, dx):
    """dx[t] = sum_j da[rows[t,j]]: moe_dispatch_bf16's gradient."""
    return moe_combine_bf16(da, rows, dx)


def moe_combine_bf16_backward(dout, o, rows, weights=None, do=None, dweights=None, m_indices=None):
    """Gradients of moe_combine_bf16 from dout bf16 [T,H] (see include/dg.h):
    writes those of do bf16, of o's shape (may be o), and dweights fp32 [T,k]
    that are given and returns both.  With m_indices (contiguous layout) the
    padding rows of do become zeros."""
    shape, dev = _matrix(dout, "dout", _current_device)
    t, h = shape
    dp, ldd = _rows(dout, _BF16, shape, dev, "dout")
    op, m = _layout(o, _BF16, h, dev, "o")
    rp, k = _slots(rows, t, dev)
    st = _lib.dg_moe_combine_bf16_backward(
        dp, ldd, op, rp, _optional(weights, _F32, (t, k), dev, "weights"),
        _optional(m_indices, _I32, (m,), dev, "m_indices"), _optional(do, _BF16, o.shape, dev, "do"),
        _optional(dweights, _F32, (t, k), dev, "dweights"), t, k, h, m, _stream_of(dev))
    if st:
        raise DGError(st, "dg_moe_combine_bf16_backward")
    return do, dweights


# ------------------------------------------------------ page-style names ---

def gemm_fp8_fp8_bf16_nt(lhs, rhs, out):
    return dg_gemm_fp8_nt(lhs[0], lhs[1], rhs[0], rhs[1], out)


def gemm_fp8_fp8_bf16_nt_ue8m0(lhs, rhs, out):
    """Power-of-two scales as fp32 values, or packed UE8M0 (int32 words)."""
    if lhs[1].dtype == torch.int32:
        return dg_gemm_fp8_nt_ue8m0_packed(lhs[0], lhs[1], rhs[0], rhs[1], out)
    return dg_gemm_fp8_nt_ue8m0(lhs[0], lhs[1], rhs[0], rhs[1], out)


def gemm_bf16_bf16_bf16_nt(lhs, rhs, out):
    return dg_gemm_bf16_nt(lhs, rhs, out)


def m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(lhs, rhs, out, m_indices):
    """fp32 scales, or packed UE8M0 (int32 words)."""
    if lhs[1].dtype == torch.int32:
        return dg_grouped_fp8_contiguous_ue8m0_packed(lhs[0], lhs[1], rhs[0], rhs[1], out, m_indices)
    return dg_grouped_fp8_contiguous(lhs[0], lhs[1], rhs[0], rhs[1], out, m_indices)


def m_grouped_gemm_fp8_fp8_fp8_nt_contiguous_swiglu(lhs, rhs, m_indices):
    """First expert linear layer + SwiGLU + 1x128 re-quantise: returns the
    second layer's operand (fp8 [M_total,I], fp32 scales [M_total,I/128]);
    rows of padding (-1) are left as torch.empty gives them."""
    m_total = lhs[0].shape[0]
    i = rhs[0].shape[1] // 2
    dev = lhs[0].device
    return dg_grouped_fp8_contiguous_swiglu(
        lhs[0], lhs[1], rhs[0], rhs[1], torch.empty((m_total, i), dtype=FP8, device=dev),
        torch.empty((m_total, i // 128), dtype=torch.float32, device=dev), m_indices)


def m_grouped_gemm_bf16_bf16_bf16_nt_contiguous(lhs, rhs, out, m_indices):
    return dg_grouped_bf16_contiguous(lhs, rhs, out, m_indices)


def m_grouped_gemm_bf16_bf16_bf16_nt_masked(lhs, rhs, out, masked_m):
    return dg_grouped_bf16_masked(lhs, rhs, out, masked_m)


def m_grouped_gemm_fp8_fp8_bf16_nt_masked(lhs, rhs, out, masked_m):
    """fp32 scales, or packed UE8M0 (int32 words)."""
    if lhs[1].dtype == torch.int32:
        return dg_grouped_fp8_masked_ue8m0_packed(lhs[0], lhs[1], rhs[0], rhs[1], out, masked_m)
    return dg_grouped_fp8_masked(lhs[0], lhs[1], rhs[0], rhs[1], out, masked_m)


def wgrad_gemm_fp8_fp8_fp32_nt(lhs, rhs, out):
    return dg_wgrad_fp8_nt(lhs[0], lhs[1], rhs[0], rhs[1], out)


def k_grouped_wgrad_gemm_fp8_fp8_fp32_nt(lhs, rhs, out, ks):
    return dg_k_grouped_wgrad_fp8_nt(lhs[0], lhs[1], rhs[0], rhs[1], out, ks)


def quantize_fp8_1x128(x):
    """Activations: (fp8 [M,K], fp32 scales [M,K/128]) for the GEMM calls above."""
    m, k = x.shape
    return dg_quantize_fp8_1x128(x, torch.empty((m, k), dtype=FP8, device=x.device),
                                 torch.empty((m, k // 128), dtype=torch.float32, device=x.device))


def quantize_fp8_128x128(x):
    """Weights: (fp8 [N,K], fp32 scales [ceil(N/128),K/128])."""
    n, k = x.shape
    return dg_quantize_fp8_128x128(x, torch.empty((n, k), dtype=FP8, device=x.device),
                                   torch.empty(((n + 127) // 128, k // 128), dtype=torch.float32, device=x.device))


def quantize_fp8_1x128_ue8m0(x):
    """Activations with power-of-two scales: (fp8 [M,K], packed UE8M0 int32 [M,ceil(K/512)])."""
    m, k = x.shape
    return dg_quantize_fp8_1x128_ue8m0(x, torch.empty((m, k), dtype=FP8, device=x.device),
                                       torch.empty((m, (k // 128 + 3) // 4), dtype=torch.int32, device=x.device))


def quantize_fp8_128x128_ue8m0(x):
    """Weights with power-of-two scales: (fp8 [N,K], packed UE8M0 int32 [ceil(N/128),ceil(K/512)])."""
    n, k = x.shape
    return dg_quantize_fp8_128x128_ue8m0(x, torch.empty((n, k), dtype=FP8, device=x.device),
                                         torch.empty(((n + 127) // 128, (k // 128 + 3) // 4), dtype=torch.int32,
                                                     device=x.device))


def quantize_fp8_1x128_transposed(x):
    """Weight-gradient operand from x [T,F]: (fp8 [F,T], fp32 scales [F,T/128])."""
    t, f = x.shape
    return dg_quantize_fp8_1x128_transposed(x, torch.empty((f, t), dtype=FP8, device=x.device),
                                            torch.empty((f, t // 128), dtype=torch.float32, device=x.device))


def quantize_int8_rows(x):
    """Operand of gemm_int8_nt_epilogue from x bf16 or fp32 [M,K]: (int8 [M,K], fp32 scales [M])."""
    return dg_quantize_int8_rows(x, torch.empty(x.shape, dtype=torch.int8, device=x.device),
                                 torch.empty(x.shape[0], dtype=torch.float32, device=x.device))


def swiglu_quantize_fp8_1x128(c):
    """Second-GEMM operand from the first GEMM's bf16 output c [M,2I]:
    (fp8 silu(gate)*up [M,I], fp32 scales [M,I/128])."""
    m, i2 = _even_width(c)
    i = i2 // 2
    return dg_swiglu_quantize_fp8_1x128(c, torch.empty((m, i), dtype=FP8, device=c.device),
                                        torch.empty((m, i // 128), dtype=torch.float32, device=c.device))
