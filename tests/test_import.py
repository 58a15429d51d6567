"""The package without the MX operators' binding (not built, or built against
another torch): the codecs, which need only libw4.so, import and work; the MX
operators say what to build."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "weight_only_bit_unpack_amd"

PROGRAM = f"""
import torch
import {PKG} as w4
assert w4.w4_group_size(w4.W4_LUT16) == 64
for call in (lambda: w4.w4_mx_quantize(torch.zeros(4, 64)),
             lambda: w4.w4_mx_dequant(torch.zeros(4, 32), torch.zeros(4, 2)),
             lambda: w4.w4_mx_rmsnorm(torch.zeros(4, 64), torch.zeros(64)),
             lambda: w4.w4_mx_linear(*[torch.zeros(4, 64)] * 4),
             lambda: w4.w4_mx_grouped_linear(*[torch.zeros(4, 64)] * 5)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and "_w4mx" in str(e), e
    else:
        raise AssertionError("no error")
print("imported")
"""


@pytest.mark.parametrize("binding", ["missing", "not a library"])
def test_codecs_import_without_the_mx_binding(tmp_path, binding):
    pkg = tmp_path / PKG
    pkg.mkdir()
    src = os.path.join(ROOT, PKG)
    for f in os.listdir(src):
        if f.endswith(".py") or f == "libw4.so":
            shutil.copy(os.path.join(src, f), pkg / f)
    if binding != "missing":
        (pkg / "_w4mx.so").write_bytes(b"\x7fELF, but not one that loads")
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0 and "imported" in r.stdout, r.stdout + r.stderr


def test_build_without_a_host_compiler_keeps_the_library(tmp_path, monkeypatch):
    """What is missing is named; libw4.so was linked before."""
    import importlib.util
    spec = importlib.util.spec_from_file_location("w4_build", os.path.join(ROOT, PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    monkeypatch.setattr(b, "BINDING_LIB", str(tmp_path / "_w4mx.so"))
    monkeypatch.setattr(b, "CXX", str(tmp_path / "no-such-compiler"))
    with pytest.raises(RuntimeError, match="codecs.*libw4.so.*is built"):
        b._build_binding()
