"""CPU tests of what the calls on bf16 rows and MXFP4 weights refuse (these return
before any HIP call), and of the same layer built for the host under
AddressSanitizer and UndefinedBehaviorSanitizer."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
INVAL, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4
POINTERS = "w ws x y gu dy dx dh dgu".split()


@pytest.fixture(scope="module")
def lib():
    import weight_only_bit_unpack_amd as m
    return m._lib


def P(v):
    return None if v is None else ctypes.c_void_p(v)


def caller(fn, names, ok):
    names = names.split()

    def call(**kw):
        a = {**ok, **kw}
        return fn(*[P(a[n]) if n in POINTERS else a[n] for n in names], None)
    return call


def sizes_and_pointers(call, operands, out):
    """What all four calls refuse."""
    assert call(n=-1) == INVAL and call(m=-1) == INVAL and call(k=-64) == INVAL
    assert call(k=16) == SHAPE and call(k=4194304 + 32) == SHAPE and call(m=1 << 31) == SHAPE
    assert call(n=4194304 + 1) == SHAPE and call(n=2 ** 62) == SHAPE
    assert call(dt=2) == UNSUP and call(dt=-1) == UNSUP
    for p in operands + [out]:
        assert call(**{p: None}) == INVAL, p
    for p in operands:
        assert call(**{p: 8}) == ALIGN, p
    assert call(**{out: 18}) == ALIGN and call(**{out: 17}, dt=1) == ALIGN


def test_linear(lib):
    call = caller(lib.w4_mx_linear_bf16, "n k w ws x m y dt", dict(n=16, k=64, w=16, ws=16, x=16, m=3, y=16, dt=0))
    sizes_and_pointers(call, ["w", "ws", "x"], "y")
    assert call(m=0, x=None, y=None) == 0 and call(n=0, w=None, ws=None, y=None) == 0


def test_gated(lib):
    call = caller(lib.w4_mx_gated_linear, "act n k w ws x m gu y dt",
                  dict(act=0, n=16, k=64, w=16, ws=16, x=16, m=3, gu=16, y=16, dt=0))
    sizes_and_pointers(call, ["w", "ws", "x"], "y")
    assert call(act=-1) == INVAL and call(act=3) == INVAL
    assert call(n=2097152 + 1) == SHAPE                # of 2 n rows
    assert call(gu=17) == ALIGN
    assert call(m=0, x=None, y=None) == 0 and call(n=0, w=None, ws=None, y=None) == 0


def test_linear_grad(lib):
    call = caller(lib.w4_mx_linear_grad, "n k w ws dy m dx dt", dict(n=16, k=64, w=16, ws=16, dy=16, m=3, dx=16, dt=0))
    sizes_and_pointers(call, ["w", "ws", "dy"], "dx")
    assert call(m=0, dy=None, dx=None) == 0 and call(k=0, w=None, ws=None, dx=None) == 0


def test_gated_grad(lib):
    call = caller(lib.w4_mx_gated_linear_grad, "act n k w ws dh gu m dgu dx dt",
                  dict(act=0, n=16, k=64, w=16, ws=16, dh=16, gu=16, m=3, dgu=16, dx=16, dt=0))
    sizes_and_pointers(call, ["w", "ws", "dh", "gu", "dgu"], "dx")
    assert call(act=-1) == INVAL and call(act=3) == INVAL
    assert call(n=2097152 + 1) == SHAPE
    assert call(m=0, dh=None, gu=None, dgu=None, dx=None) == 0
    assert call(n=0, k=0, w=None, ws=None, dx=None) == 0


def test_more_than_a_launch(lib):
    """More blocks than 2^32 threads hold are refused, not cut."""
    A = ctypes.c_void_p(4096)
    n, m = 4194304, 2 ** 31 - 1
    assert lib.w4_mx_linear_bf16(n, 32, A, A, A, m, A, 1, None) == SHAPE
    assert lib.w4_mx_gated_linear(0, n // 2, 32, A, A, A, m, None, A, 1, None) == SHAPE
    assert lib.w4_mx_linear_grad(32, n, A, A, A, m, A, 1, None) == SHAPE
    assert lib.w4_mx_gated_linear_grad(0, 32, n, A, A, A, A, m, A, A, 1, None) == SHAPE


def test_every_kernel_is_taken_by_some_product(lib):
    """Each tile, whole and with its last ones in parts, and each few-row shape, on the
    card's 256 compute units."""
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    f = lib.w4_mx_bf16_kernel_of
    f.argtypes, f.restype = [i32, i64, i64, i64], i32
    ms = [1, 16, 17, 64, 130, 333, 700, 1500, 2050, 4100]
    ns = [96, 513, 1100, 2730, 4100, 5500, 11008, 33000]
    ks = [64, 256, 1024, 2272, 4096, 11008, 32768]
    for kind in (0, 1, 2):
        seen = {f(kind, n, k, m) for m in ms for n in ns for k in ks}
        plain, cut = {s for s in seen if s < 1024}, {s - 1024 for s in seen if 1024 <= s < 4096}
        assert {s % 16 for s in plain} == set(range(5)), kind
        assert {s // 16 for s in plain} >= {1, 2, 3, 4, 6, 8, 12}, kind
        assert {s % 16 for s in cut} >= {0, 2}, kind
        assert {s - 4096 for s in seen if s >= 4096} == (set() if kind == 2 else {0, 1, 2}), kind


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the HIP headers")
def test_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "mx_bf16_api_check")
    csrc = os.path.join(ROOT, "weight_only_bit_unpack_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(csrc, "w4_mx_bf16_api.cpp"), os.path.join(HERE, "mx_bf16_api_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0 and "mx_bf16_api_check ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
