"""The host code of the linear layer and the few-token MoE layer under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: plans over sizes
and compute-unit counts, held against what the kernels assume, with the HIP
runtime and the launches replaced by functions that look at their arguments."""
from __future__ import annotations

import os

from tests.test_host_sanitizers import CSRC, HIPCC, HOST_SAN, ROOT, SAN, _check_clean, _run


def test_plans_and_calls_under_sanitizers(tmp_path):
    exe = str(tmp_path / "linear_driver")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", *HOST_SAN, "-pthread",
          "-I", os.path.join(ROOT, "include"), "-o", exe, *(os.path.join(CSRC, s) for s in
                                                          ("dg_api.hip", "dg_shapes.hip", "dg_linear.hip", "dg_moe.hip")),
          os.path.join(SAN, "linear_driver.hip")])
    _check_clean(_run([exe], timeout=120))
