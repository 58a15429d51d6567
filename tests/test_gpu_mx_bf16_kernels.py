"""Every kernel of the products of bf16 rows and MXFP4 weights by name, whatever the
plan would take, through w4_mx_bf16_product_on: each tile, number of parts and few-row
shape, on operands whose sums are exact whatever their order (compared bit for bit)."""

import ctypes

import numpy as np
import pytest
import torch

from tests.gpu_util import report
from tests.test_gpu_mx_bf16 import (BF16, F32, canary, dev, edges_kept, exact_rows, exact_weight, gated_within, same)

pytestmark = pytest.mark.gpu

FORWARD, GATED, BACKWARD = 0, 1, 2
TAIL, FEW = 1024, 4096


@pytest.fixture(scope="module")
def lib():
    import weight_only_bit_unpack_amd as m
    i, j, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    m._lib.w4_mx_bf16_product_on.argtypes = [i, i, i, j, j, p, p, p, j, p, p, i, p]
    return m._lib


def on(lib, kernel, kind, n, k, wq, ws, x, gu, y):
    return lib.w4_mx_bf16_product_on(kernel, kind, 0, n, k, wq.data_ptr(), ws.data_ptr(), x.data_ptr(), x.shape[0],
                                     None if gu is None else gu.data_ptr(), y.data_ptr(), int(y.dtype == BF16),
                                     torch.cuda.current_stream().cuda_stream)


def check(lib, kernel, kind, m, n, k, dtype):
    g = np.random.default_rng(m + n + k)
    wq, ws, w = exact_weight(g, 2 * n if kind == GATED else n, k)
    x = exact_rows(g, m, n if kind == BACKWARD else k)
    out = k if kind == BACKWARD else n
    buf, y = canary(m, out, dtype)
    if kernel < TAIL and kernel >= 32:                   # a tile is cut into parts, at most 1024 in all
        rows, cols = [(256, 256), (128, 256), (128, 128), (64, 128), (32, 64)][kernel % 16]
        cols = cols // 2 if kind == GATED else cols
        if -(-m // rows) * -(-out // cols) * (kernel // 16) > 1024:
            assert on(lib, kernel, kind, n, k, wq, ws, dev(x), None, y) != 0
            return
    if kind == GATED:
        x = x / 64 * 2.0 ** -int(np.log2(k) / 2)
        gbuf, gu = canary(m, 2 * n, BF16)
        assert on(lib, kernel, kind, n, k, wq, ws, dev(x), gu, y) == 0
        want = x @ w.T
        same(gu, want)
        gated_within(y, want[:, :n], want[:, n:], "silu")
        assert edges_kept(gbuf, m, 2 * n)
    else:
        assert on(lib, kernel, kind, n, k, wq, ws, dev(x), None, y) == 0
        same(y, x @ w if kind == BACKWARD else x @ w.T)
    assert edges_kept(buf, m, out)


# (m, n, k): one row, one tile and one beside, several tiles, short and long sums that
# end inside a step, counts of steps around the steps in flight
SIZES = [(1, 40, 64), (33, 72, 96), (70, 136, 160), (129, 264, 224), (257, 520, 288), (300, 200, 1056),
         (40, 1032, 416), (520, 1288, 352)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", [FORWARD, GATED, BACKWARD])
@pytest.mark.parametrize("tile", range(5))
def test_tiles_and_parts(lib, tile, kind, dtype):
    for m, n, k in SIZES:
        steps = ((n if kind == BACKWARD else k) + 63) // 64
        for parts in (1, 2, 3, 5, 16):
            if parts > steps:
                continue
            report("mx_bf16_kernel", tile=tile, kind=kind, parts=parts, m=m, n=n, k=k, dtype=dtype)
            check(lib, 16 * parts + tile, kind, m, n, k, dtype)


@pytest.mark.parametrize("kind", [FORWARD, GATED, BACKWARD])
@pytest.mark.parametrize("tile", range(4))
def test_last_tiles_in_parts(lib, tile, kind):
    """Some tiles whole and the others cut, in one launch."""
    for m, n, k in ((600, 2312, 416), (1100, 520, 1312)):
        for parts in (2, 3, 4):
            report("mx_bf16_tail", tile=tile, kind=kind, parts=parts, m=m, n=n, k=k)
            check(lib, TAIL + 16 * parts + tile, kind, m, n, k, BF16)


@pytest.mark.parametrize("kind", [FORWARD, BACKWARD])
@pytest.mark.parametrize("tile", range(5))
def test_every_step_count(lib, tile, kind):
    """Sums of 1 to 14 steps, whole and ending inside one."""
    for steps in range(1, 15):
        for over in (-32, 0) if kind == FORWARD else (-56, -8, 0):
            size = 64 * steps + over
            if size > 0:
                report("mx_bf16_steps", tile=tile, kind=kind, terms=size)
                check(lib, 16 + tile, kind, 70, *((96, size) if kind == FORWARD else (size, 96)), F32)


@pytest.mark.parametrize("kind", [FORWARD, GATED])
@pytest.mark.parametrize("shape", range(3))
def test_few_rows(lib, shape, kind):
    for m in (1, 2, 3, 4, 5, 8, 9, 16):
        for n, k in ((1, 32), (17, 96), (40, 256), (130, 288), (64, 2080), (33, 4128)):
            report("mx_bf16_few_rows", shape=shape, kind=kind, m=m, n=n, k=k)
            check(lib, FEW + shape, kind, m, n, k, BF16 if m % 2 else F32)


def test_parts_again_and_again(lib):
    """The counts are back at zero after each launch: the same tiles in parts many times
    over, mixed with other numbers of parts, with the same bits every time."""
    g = np.random.default_rng(9)
    m, n, k = 100, 200, 2080
    wq, ws, w = exact_weight(g, n, k)
    x = exact_rows(g, m, k)
    xd, want = dev(x), x @ w.T
    for _ in range(30):
        for kernel in (16 * 16 + 4, 16 * 3 + 2, 16 * 2 + 0, 16 * 7 + 3, TAIL + 16 * 2 + 4):
            y = torch.full((m, n), float("nan"), device="cuda")
            assert on(lib, kernel, FORWARD, n, k, wq, ws, xd, None, y) == 0
            same(y, want)


def test_what_does_not_fit_is_refused(lib):
    u8 = torch.zeros((64, 32), dtype=torch.uint8, device="cuda")
    x, y = torch.zeros((17, 64), dtype=BF16, device="cuda"), torch.full((17, 64), 7.0, device="cuda")
    for kernel, kind, n in ((16 + 5, FORWARD, 64), (16 * 17, FORWARD, 64), (0, FORWARD, 64), (32, FORWARD, 64),
                            (FEW, FORWARD, 64), (FEW, BACKWARD, 64), (FEW + 3, GATED, 32), (16, BACKWARD, 63),
                            (16, 3, 64), (-16, FORWARD, 64)):
        assert on(lib, kernel, kind, n, 64, u8, u8, x, None, y) != 0, (kernel, kind, n)
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
