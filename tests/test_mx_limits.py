"""CPU tests of what the MX calls refuse for size: these return before any HIP call."""

import ctypes

import pytest

SHAPE = 2


@pytest.fixture(scope="module")
def lib():
    import weight_only_bit_unpack_amd as m
    return m._lib


A = ctypes.c_void_p(4096)


@pytest.mark.parametrize("fmt", [0, 1])
def test_products_beyond_a_launch(lib, fmt):
    """More blocks than 2^32 threads hold are refused, not cut."""
    n = 4194304
    # many rows a weight, few rows a weight, one weight
    assert lib.w4_mx_grouped_linear(fmt, 2048, n, 32, A, A, 64, A, A, 20000, A, A, A, 1, None) == SHAPE
    assert lib.w4_mx_grouped_linear(fmt, 2048, n, 32, A, A, 64, A, A, 5000, A, A, A, 1, None) == SHAPE
    assert lib.w4_mx_linear(fmt, 64, 32, A, A, A, A, 2 ** 31 - 1, A, 1, None) == SHAPE


def test_every_kernel_is_taken_by_some_product(lib):
    """Each tile, each number of parts of k and each shape of the few-row kernel, for
    either format, on the card's 256 compute units."""
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    f = lib.w4_mx_kernel_of
    f.argtypes, f.restype = [i32, i32, i64, i64, i64], i32
    ms = [1, 16, 17, 33, 64, 129, 200, 513, 700, 1100, 2050, 4100, 8200]
    ns = [96, 513, 1100, 2050, 2900, 4100, 8200, 33000]
    ks = [224, 1024, 2272, 4096, 8192, 16384, 32768]
    for fmt in (0, 1):
        for experts in (0, 5, 64):
            seen = {f(fmt, experts, n, k, m) for m in ms for n in ns for k in ks}
            if experts == 0:
                assert {s % 16 for s in seen if s < 256} == set(range(5)), fmt
                assert {s // 16 for s in seen if s < 256} == {1, 2, 4, 8}, fmt
                assert {s - 256 for s in seen if s >= 256} >= {0, 1}, fmt
            elif experts == 5:
                assert {s for s in seen if s < 256} == {16 + t for t in range(5)}, fmt
            else:
                assert {s - 256 for s in seen if s >= 256} == {0, 1, 2}, fmt
