"""CPU tests of the MX calls' argument validation (these calls return before
any HIP call is made), and of the same layer built for the host under
AddressSanitizer and UndefinedBehaviorSanitizer."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
INVAL, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    import weight_only_bit_unpack_amd as m
    return m._lib


def P(v):
    return None if v is None else ctypes.c_void_p(v)


def caller(fn, names, ok):
    def call(**kw):
        a = {**ok, **kw}
        return fn(*[P(a[n]) if n in "x q s out res gamma ro y w ws xs off idx".split() else a[n] for n in names],
                  None)
    return call


def test_quantize_and_dequant(lib):
    names = ["fmt", "rows", "k", "x", "dt", "q", "s"]
    call = caller(lib.w4_mx_quantize, names, dict(fmt=0, rows=4, k=64, x=16, dt=1, q=16, s=16))
    assert call(fmt=2) == INVAL and call(fmt=-1) == INVAL
    assert call(rows=-1) == INVAL and call(k=-32) == INVAL
    assert call(k=48) == SHAPE and call(rows=1 << 60) == SHAPE
    assert call(dt=3) == UNSUP
    assert call(x=None) == INVAL and call(q=None) == INVAL and call(s=None) == INVAL
    assert call(x=8) == ALIGN and call(q=4) == ALIGN and call(s=2) == ALIGN
    assert call(rows=0, x=None, q=None, s=None) == 0
    assert call(k=0, x=None, q=None, s=None) == 0
    names = ["fmt", "rows", "k", "q", "s", "out", "dt"]
    call = caller(lib.w4_mx_dequant, names, dict(fmt=1, rows=4, k=64, q=16, s=16, out=16, dt=1))
    assert call(fmt=2) == INVAL and call(rows=-1) == INVAL and call(k=33) == SHAPE
    assert call(dt=2) == UNSUP                       # fp16 could not hold the values
    assert call(out=None) == INVAL and call(out=8) == ALIGN and call(q=8) == ALIGN
    assert call(rows=0, q=None, s=None, out=None) == 0


def test_rmsnorm(lib):
    names = ["fmt", "rows", "k", "x", "res", "gamma", "dt", "eps", "ro", "y", "q", "s"]
    call = caller(lib.w4_mx_rmsnorm, names, dict(fmt=1, rows=4, k=64, x=16, res=16, gamma=16, dt=1, eps=1e-5,
                                                 ro=16, y=16, q=16, s=16))
    assert call(fmt=5) == INVAL and call(rows=-1) == INVAL and call(k=40) == SHAPE
    assert call(rows=1 << 31, k=32) == SHAPE
    assert call(dt=7) == UNSUP
    assert call(eps=-1.0) == INVAL and call(eps=float("nan")) == INVAL and call(eps=float("inf")) == INVAL
    assert call(x=None) == INVAL and call(gamma=None) == INVAL and call(ro=None) == INVAL
    assert call(y=None, q=None) == INVAL and call(s=None) == INVAL
    for n in ("x", "res", "gamma", "ro", "y", "q", "s"):
        assert call(**{n: 8}) == ALIGN, n
    assert call(rows=0, x=None, gamma=None, ro=None, y=None, q=None, s=None) == 0


def test_linear(lib):
    names = ["fmt", "n", "k", "w", "ws", "x", "xs", "m", "y", "dt"]
    call = caller(lib.w4_mx_linear, names, dict(fmt=1, n=16, k=64, w=16, ws=16, x=16, xs=16, m=3, y=16, dt=0))
    assert call(fmt=2) == INVAL and call(n=-1) == INVAL and call(m=-1) == INVAL and call(k=-64) == INVAL
    assert call(k=16) == SHAPE and call(k=4194304 + 32) == SHAPE and call(m=1 << 31) == SHAPE
    assert call(m=2 ** 31 - 1, n=2 ** 31 - 1) == SHAPE
    assert call(dt=2) == UNSUP
    for n in ("w", "ws", "x", "xs", "y"):
        assert call(**{n: None}) == INVAL, n
    for n in ("w", "ws", "x", "xs"):
        assert call(**{n: 8}) == ALIGN, n
    assert call(y=18) == ALIGN and call(y=17, dt=1) == ALIGN
    assert call(m=0, x=None, xs=None, y=None) == 0
    assert call(n=0, w=None, ws=None, y=None) == 0


def test_grouped_linear(lib):
    names = ["fmt", "E", "n", "k", "w", "ws", "tokens", "x", "xs", "rows", "off", "idx", "y", "dt"]
    call = caller(lib.w4_mx_grouped_linear, names, dict(fmt=1, E=4, n=16, k=64, w=16, ws=16, tokens=3, x=16, xs=16,
                                                        rows=6, off=16, idx=16, y=16, dt=0))
    assert call(fmt=2) == INVAL and call(E=-1) == INVAL and call(tokens=-1) == INVAL and call(rows=-1) == INVAL
    assert call(E=4097) == SHAPE and call(k=96 + 16) == SHAPE and call(idx=None) == SHAPE
    assert call(rows=2 ** 31 - 1, n=2 ** 31 - 1) == SHAPE
    assert call(dt=2) == UNSUP
    for n in ("w", "ws", "x", "xs", "off", "y"):
        assert call(**{n: None}) == INVAL, n
    for n in ("w", "ws", "x", "xs"):
        assert call(**{n: 24}) == ALIGN, n
    assert call(off=18) == ALIGN and call(idx=18) == ALIGN and call(y=18) == ALIGN
    assert call(rows=0, x=None, xs=None, off=None, idx=None, y=None, tokens=0) == 0


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP headers")
def test_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "mx_api_check")
    csrc = os.path.join(ROOT, "weight_only_bit_unpack_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(csrc, "w4_mx_api.cpp"), os.path.join(HERE, "mx_api_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0 and "mx_api_check ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
