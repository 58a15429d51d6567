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
