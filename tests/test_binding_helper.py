"""The binding without its native helper (another torch or Python, no host
compiler), and the structures that it packs itself, on the CPU."""
from __future__ import annotations

import importlib.util
import os
import re
import struct
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "moe_grouped_gemm_x128_amd")

WITHOUT = """
import sys, types, warnings
name = "moe_grouped_gemm_x128_amd._tensors"
if {other_torch}:
    sys.modules[name] = m = types.ModuleType(name)
    m.built_with = "0.1"
    import importlib.machinery
    m.__spec__ = importlib.machinery.ModuleSpec(name, None)
else:
    sys.modules[name] = None  # importing it raises ImportError
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import moe_grouped_gemm_x128_amd as dg
assert dg._tensors is None
assert any("native helper" in str(w.message) for w in seen), [str(w.message) for w in seen]
import torch
x = torch.zeros((4, 256), dtype=torch.bfloat16)
for call in (lambda: dg.rmsnorm_bf16(x, None, x), lambda: dg.gemm_int8_nt_epilogue((x, x), (x, x), x),
             lambda: dg.moe_combine_bf16(x, x, x)):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e)
    else:
        raise AssertionError("a CPU tensor was taken")
for f in (dg._whole, dg._rows):
    for t, kind in ((3, TypeError), (x.float(), TypeError), (x[:2], ValueError), (x, ValueError)):
        try:
            f(t, torch.bfloat16, (4, 256), 0, "x")
        except kind as e:
            assert str(e).startswith("x ")
        else:
            raise AssertionError(str(t))
print(dg.version())
"""


@pytest.mark.parametrize("other_torch", [False, True])
def test_package_loads_without_the_helper(other_torch):
    out = subprocess.run([sys.executable, "-c", WITHOUT.format(other_torch=other_torch)], cwd=ROOT, capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr


def builder(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(PACKAGE, "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_library_is_built_where_the_helper_cannot_be(tmp_path, monkeypatch, capsys):
    b = builder("_build_for_test")
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "TENSORS", str(tmp_path / "_tensors.so"))
    monkeypatch.setattr(b, "CXX", str(tmp_path / "no-compiler"))
    monkeypatch.setattr(b, "_hipcc", lambda args, verbose: open(args[args.index("-o") + 1], "w").close())
    (tmp_path / "_tensors.so").write_text("of older sources")
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.TENSORS)
    assert "native helper was not built" in capsys.readouterr().err


def test_helper_is_named_for_this_python():
    assert re.search(r"cpython-3\d+", os.path.basename(builder("_build_for_test").TENSORS))


def test_packed_structures_are_the_header_s(tmp_path):
    """The binding's struct formats against the compiler's layout of dg_norm and dg_epilogue."""
    import moe_grouped_gemm_x128_amd as dg

    fields = {"dg_norm": ["x", "ld_x", "residual", "ld_residual", "weight", "weight_type", "eps", "sum", "ld_sum", "rstd"],
              "dg_epilogue": ["bias", "bias_type", "activation", "residual", "ld_residual", "pre", "ld_pre"]}
    src = '#include <stddef.h>\n#include <stdio.h>\n#include "dg.h"\nint main(void) {\n'
    for s, names in fields.items():
        src += "".join(f'printf("%zu ", offsetof({s}, {n}));\n' for n in names) + f'printf("%zu\\n", sizeof({s}));\n'
    (tmp_path / "layout.c").write_text(src + "return 0;\n}\n")
    exe = str(tmp_path / "layout")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(builder("_build_for_test").HIPCC)))
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__=1", f"-I{ROOT}/include", f"-I{rocm}/include",
                    str(tmp_path / "layout.c"), "-o", exe], check=True)
    got = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()
    for line, pack in zip(got, (dg._norm_fields, dg._epilogue_fields)):
        form = pack.__self__.format
        offsets = [struct.calcsize(form[:i]) + (-struct.calcsize(form[:i])) % struct.calcsize(form[i])
                   for i in range(len(form))]
        assert [int(v) for v in line.split()] == offsets + [struct.calcsize(form)]
