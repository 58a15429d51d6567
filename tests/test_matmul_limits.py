"""CPU tests of what the codec matrix calls refuse for size: work for 2^32 threads
or more, which one launch does not hold, before any HIP call is made."""

import ctypes

import pytest

SHAPE = 2
A = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def w4():
    import weight_only_bit_unpack_amd as m
    return m


@pytest.mark.parametrize("codec", [0, 1, 2, 3, 4, 5])
def test_gemv_and_gemm(w4, codec):
    call = lambda f, n, k, m: f(codec, n, k, A, A, A, A, m, A, 1, None)
    assert call(w4._lib.w4_gemv, 2 ** 30 + 64, 64, 1) == SHAPE          # 64 rows a block of 256
    assert call(w4._lib.w4_gemv, 2 ** 30 + 64, 64, 4) == SHAPE
    assert call(w4._lib.w4_linear, 2 ** 30 + 64, 64, 4) == SHAPE
    m = 65535 * 128
    assert call(w4._lib.w4_gemm, 64, 8192, m) == SHAPE                  # packing x: eight values a thread
    assert call(w4._lib.w4_gemm, 2 ** 16, 64, m) == SHAPE               # 128 x 256 outputs a block of 512
    assert call(w4._lib.w4_linear, 2 ** 16, 64, m) == SHAPE


def test_batched_plan(w4):
    a = lambda n: (w4.W4Problem * 1)(w4.W4Problem(4096, 4096, 4096, 4096, 4096, n, 64, 0))
    info = w4.W4BatchInfo()
    plan = lambda n: w4._lib.w4_gemv_batched_plan(0, 1, 0, a(n), 1, ctypes.byref(info))
    assert plan(2 ** 30) == SHAPE and plan(2 ** 30 - 64) == 0
    assert info.total_tiles == 2 ** 24 - 1
    info.total_tiles = 2 ** 24
    assert w4._lib.w4_gemv_batched(0, 1, 0, A, ctypes.byref(info), None) == SHAPE
