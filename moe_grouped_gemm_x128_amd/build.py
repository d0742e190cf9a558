"""Build the gfx950 HIP library (libdg_mi355x.so) in-tree with hipcc, and the
binding's native helper (_tensors) with the host compiler.  The binding works
without the helper, only slower, so a failure of that part is a warning.

    python moe_grouped_gemm_x128_amd/build.py        # or build() from Python

Packed-fp32 instructions are disabled for the device code (the flag only
concerns the gfx950 pass; hipcc's host pass warns that it does not know it).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdg_mi355x.so")
SOURCES = ["dg_api.hip", "dg_shapes.hip", "dg_kernels.hip", "dg_quant.hip", "dg_noalloc.hip", "dg_moe.hip",
           "dg_linear.hip", "dg_linear_rows.hip", "dg_linear_gemm.hip", "dg_linear_int8.hip", "dg_linear_int8_gemm.hip",
           "dg_norm.hip", "dg_moe_rows.hip"]
# (named for this Python: another one does not take it for its own)
TENSORS = os.path.join(HERE, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))
CXX = os.environ.get("CXX", "g++")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # keep MFMA results in VGPRs: the promotion FMAs read them directly
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    "-I", os.path.join(ROOT, "include"),
]


def _hipcc(args, verbose):
    cmd = [HIPCC, *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed with exit code {res.returncode}")


def build_tensors(verbose: bool = False) -> str:
    """Compile csrc/dg_tensors.cpp against the installed torch."""
    import torch
    from torch.utils import cpp_extension

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TENSORS + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DDG_TORCH_VERSION="{torch.__version__}"', "-D__HIP_PLATFORM_AMD__=1",
           *(f"-I{p}" for p in [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
                                os.path.join(ROOT, "include"),
                                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "include")]),
           os.path.join(CSRC, "dg_tensors.cpp"), "-o", tmp, f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{CXX} failed with exit code {res.returncode}")
    os.replace(tmp, TENSORS)
    return TENSORS


def build(verbose: bool = False, extra=None) -> str:
    """Compile every source (one hipcc each, in parallel) and link the shared
    library, then the binding's helper; always recompiles."""
    tmp = LIB + ".tmp"
    flags = [*FLAGS, *(extra or [])]
    with tempfile.TemporaryDirectory() as objs:
        out = {s: os.path.join(objs, s + ".o") for s in SOURCES}
        with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as pool:
            list(pool.map(lambda s: _hipcc([*flags, "-c", "-o", out[s], os.path.join(CSRC, s)], verbose), SOURCES))
        _hipcc([f"--offload-arch={ARCH}", "-shared", "-fPIC", *(extra or []), "-o", tmp, *out.values()], verbose)
    os.replace(tmp, LIB)
    try:
        build_tensors(verbose)
    except Exception as e:
        if os.path.exists(TENSORS):
            os.remove(TENSORS)  # (of other sources than the library's)
        sys.stderr.write(f"warning: the binding's native helper was not built ({e}): small calls take longer\n")
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
