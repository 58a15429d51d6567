"""What the library enqueues, on the CPU: libw4.so as it is built, against a stand-in
for the HIP runtime that records launches (tests/launches/fake_hip.h)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "launches")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP headers")
@pytest.mark.parametrize("check", ["counters_check", "turns_check", "throws_check"])
def test_launches(tmp_path, check):
    import weight_only_bit_unpack_amd as w4
    exe = str(tmp_path / check)
    lib = os.path.abspath(w4.LIB_PATH)
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-pthread", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(os.path.dirname(lib), "csrc"),
           os.path.join(HERE, check + ".cpp"), "-o", exe, lib, "-Wl,-rpath," + os.path.dirname(lib),
           "-rdynamic",
           "-Wl,--allow-shlib-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and check + " ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
