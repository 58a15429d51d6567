"""The library's stream workspaces, built for the host under AddressSanitizer and
UndefinedBehaviorSanitizer: calls on different streams never share a buffer."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP headers")
def test_who_shares_a_workspace(tmp_path):
    exe = str(tmp_path / "workspace_check")
    csrc = os.path.join(ROOT, "weight_only_bit_unpack_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-pthread",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(csrc, "w4_workspace.cpp"), os.path.join(HERE, "workspace_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0 and "workspace_check ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
