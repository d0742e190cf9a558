"""Build the gfx950 HIP library (libdg_mi355x.so) in-tree with hipcc.

    python moe_grouped_gemm_x128_amd/build.py        # or build() from Python

Packed-fp32 instructions are disabled for the device code (the flag only
concerns the gfx950 pass; hipcc's host pass warns that it does not know it).
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdg_mi355x.so")
SOURCES = ["dg_api.hip", "dg_shapes.hip", "dg_kernels.hip", "dg_quant.hip", "dg_noalloc.hip", "dg_moe.hip",
           "dg_linear.hip", "dg_linear_rows.hip", "dg_linear_gemm.hip"]
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


def build(verbose: bool = False, extra=None) -> str:
    """Compile every source (one hipcc each, in parallel) and link the shared
    library; always recompiles."""
    tmp = LIB + ".tmp"
    flags = [*FLAGS, *(extra or [])]
    with tempfile.TemporaryDirectory() as objs:
        out = {s: os.path.join(objs, s + ".o") for s in SOURCES}
        with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as pool:
            list(pool.map(lambda s: _hipcc([*flags, "-c", "-o", out[s], os.path.join(CSRC, s)], verbose), SOURCES))
        _hipcc([f"--offload-arch={ARCH}", "-shared", "-fPIC", *(extra or []), "-o", tmp, *out.values()], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
