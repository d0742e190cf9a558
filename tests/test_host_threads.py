"""Calls on one stream from several host threads, on the CPU: the library's
host code built with AddressSanitizer and UndefinedBehaviorSanitizer, the HIP
runtime and the kernel launches replaced by functions that write down the order
in which work reaches a stream."""
from __future__ import annotations

import os

from tests.test_host_sanitizers import CSRC, HIPCC, HOST_SAN, ROOT, SAN, _check_clean, _run


def test_split_k_calls_on_one_stream(tmp_path):
    exe = str(tmp_path / "threads_driver")
    _run([HIPCC, "--offload-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17", *HOST_SAN, "-pthread",
          "-I", os.path.join(ROOT, "include"), "-o", exe, *(os.path.join(CSRC, s) for s in
                                                          ("dg_api.hip", "dg_shapes.hip", "dg_linear.hip")),
          os.path.join(SAN, "threads_driver.hip")])
    _check_clean(_run([exe], timeout=120))
