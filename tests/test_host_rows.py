"""The host code of the norm, the sorted tokens and the INT8 layer under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: launches and plans
over sizes and compute-unit counts, held against what the kernels assume, with
the HIP runtime and the launches replaced by functions that look at their
arguments."""
from __future__ import annotations

import os

from tests.test_host_sanitizers import CSRC, HIPCC, HOST_SAN, ROOT, SAN, _check_clean, _run


def test_launches_and_calls_under_sanitizers(tmp_path):
    exe = str(tmp_path / "rows_driver")
    _run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", *HOST_SAN, "-pthread",
          "-I", os.path.join(ROOT, "include"), "-o", exe,
          *(os.path.join(CSRC, s) for s in ("dg_api.hip", "dg_shapes.hip", "dg_linear.hip", "dg_linear_int8.hip",
                                            "dg_norm.hip", "dg_moe_rows.hip")),
          os.path.join(SAN, "rows_driver.hip")])
    _check_clean(_run([exe], timeout=120))
