"""That the products of bf16 rows with MXFP4 weights hold their sums in 24 bits
throughout, on the way too: bit for bit on operands whose running sums need them, and
by the 2-norm of the error on normal data (tests/wide_sums.py; the limits are derived
there).  Through the calls, and on every kernel by name, with sums in parts and in
groups of waves."""

import numpy as np
import pytest
import torch

from oracle import mx
from tests.gpu_util import report
from tests.test_gpu_mx_bf16 import BF16, F32, bf16, dev, f64, gated_within, put, same, weight
from tests.test_gpu_mx_bf16_kernels import BACKWARD, FEW, FORWARD, GATED, TAIL, lib, on  # noqa: F401 (lib: a fixture)
from tests.wide_sums import limit, relative_error, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import weight_only_bit_unpack_amd as m
    return m


SHAPES = [(1, 64, 32), (1, 300, 4128), (3, 1000, 2048), (8, 96, 512), (16, 257, 5632), (16, 5000, 288),
          (17, 64, 2080), (40, 300, 1056), (70, 513, 640), (100, 513, 5632), (129, 1001, 992), (300, 2730, 2080),
          (600, 700, 672), (1030, 1100, 1120), (64, 96, 11008)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_wide_sums(w4, m, n, k):
    report("mx_bf16_wide", m=m, n=n, k=k)
    g = np.random.default_rng(m + n + k)
    q, s, w, x = wide(g, m, n, k)
    for dtype in (F32, BF16):
        same(w4.w4_mx_linear_bf16(dev(x), put(q), put(s), y_dtype=dtype), x @ w.T)
    q, s, w, dy = wide(g, m, n, k, back=True)
    for dtype in (F32, BF16):
        same(w4.w4_mx_linear_grad(dev(dy), put(q), put(s), dx_dtype=dtype), dy @ w)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_wide_sums_gated(w4, m, n, k):
    """Gates of a few units that are left of sums 2^20 times as large."""
    report("mx_bf16_wide_gated", m=m, n=n, k=k)
    g = np.random.default_rng(m * 3 + n + k)
    q, s, w, x = wide(g, m, 2 * n, k)
    x = x / 64 * 2.0 ** -int(np.log2(k) / 2)
    want = x @ w.T
    gu = torch.empty((m, 2 * n), dtype=BF16, device="cuda")
    y = w4.w4_mx_gated_linear(dev(x), put(q), put(s), gu=gu)
    same(gu, want)
    gated_within(y, want[:, :n], want[:, n:], "silu")


@pytest.mark.parametrize("m,n,k", [(1, 2048, 2048), (13, 4095, 5632), (16, 1000, 11008), (40, 300, 5632),
                                   (100, 513, 5632), (333, 700, 2080), (700, 1030, 11008), (1100, 5632, 512)])
def test_error_in_the_norm(w4, m, n, k):
    """fp32 outputs of normal data, both directions, and dx of the gated block's gradient."""
    report("mx_bf16_norm", m=m, n=n, k=k)
    g = np.random.default_rng(m + n * 3 + k)
    wq, ws, w = weight(g, n, k)
    x, dy = bf16(g.standard_normal((m, k))), bf16(g.standard_normal((m, n)))
    got = {"y": (w4.w4_mx_linear_bf16(dev(x), wq, ws), x @ w.T, k),
           "dx": (w4.w4_mx_linear_grad(dev(dy), wq, ws, dx_dtype=F32), dy @ w, n)}
    half = n // 2
    gu = bf16(g.standard_normal((m, 2 * half)))
    dx, dgu = w4.w4_mx_gated_linear_grad(dev(dy[:, :half].copy()), dev(gu), wq[:2 * half], ws[:2 * half], dx_dtype=F32)
    got["gated dx"] = (dx, f64(dgu) @ w[:2 * half], 2 * half)
    for name, (y, want, terms) in got.items():
        error = relative_error(f64(y), want)
        report("mx_bf16_norm", of=name, error=f"{error:.2e}", limit=f"{limit(terms, 16):.2e}")
        assert error <= limit(terms, 16), name           # (at most 16 parts)


# ------------------------------------------------------------------ every kernel by name
# (m, n, k) with sums of 5 to 33 steps, whole and ending inside one
SIZES = [(33, 72, 320), (70, 1064, 416), (129, 264, 2080)]


@pytest.mark.parametrize("kind", [FORWARD, BACKWARD])
@pytest.mark.parametrize("tile", range(5))
def test_wide_sums_on_tiles(lib, tile, kind):  # noqa: F811
    for m, n, k in SIZES:
        back = kind == BACKWARD
        g = np.random.default_rng(m + n + k + tile)
        q, s, w, x = wide(g, m, n, k, back)
        q, s, xd, want = put(q), put(s), dev(x), x @ w if back else x @ w.T
        for parts in (1, 2, 3, 8, 16):
            if parts > ((n if back else k) + 63) // 64:
                continue
            report("mx_bf16_wide_kernel", tile=tile, kind=kind, parts=parts, m=m, n=n, k=k)
            y = torch.full(want.shape, float("nan"), device="cuda")
            assert on(lib, 16 * parts + tile, kind, n, k, q, s, xd, None, y) == 0
            same(y, want)


@pytest.mark.parametrize("kind", [FORWARD, BACKWARD])
@pytest.mark.parametrize("tile", range(4))
def test_wide_sums_of_last_tiles(lib, tile, kind):  # noqa: F811
    m, n, k = 600, 2312, 416
    g = np.random.default_rng(tile)
    q, s, w, x = wide(g, m, n, k, kind == BACKWARD)
    for parts in (2, 4):
        report("mx_bf16_wide_tail", tile=tile, kind=kind, parts=parts)
        want = x @ w if kind == BACKWARD else x @ w.T
        y = torch.full(want.shape, float("nan"), device="cuda")
        assert on(lib, TAIL + 16 * parts + tile, kind, n, k, put(q), put(s), dev(x), None, y) == 0
        same(y, want)


@pytest.mark.parametrize("shape", range(3))
def test_wide_sums_of_few_rows(lib, shape):  # noqa: F811
    for m in (1, 4, 9, 16):
        for n, k in ((17, 96), (130, 2080), (33, 4128)):
            report("mx_bf16_wide_few_rows", shape=shape, m=m, n=n, k=k)
            q, s, w, x = wide(np.random.default_rng(m + n), m, n, k)
            y = torch.full((m, n), float("nan"), device="cuda")
            assert on(lib, FEW + shape, FORWARD, n, k, put(q), put(s), dev(x), None, y) == 0
            same(y, x @ w.T)


@pytest.mark.parametrize("kind", [FORWARD, GATED, BACKWARD])
@pytest.mark.parametrize("tile", range(5))
def test_error_in_the_norm_on_tiles(lib, tile, kind):  # noqa: F811
    m, n, k = 70, 1024, 1056
    g = np.random.default_rng(tile)
    rows = 2 * n if kind == GATED else n
    wq, ws, w = weight(g, rows, k)
    x = bf16(g.standard_normal((m, n if kind == BACKWARD else k)))
    for parts in (1, 4, 10):                             # (a product's parts are 1024 at most)
        y = torch.full((m, k if kind == BACKWARD else n), float("nan"), device="cuda")
        assert on(lib, 16 * parts + tile, kind, n, k, wq, ws, dev(x), None, y) == 0
        if kind == GATED:                                # silu(g) u: off by g's and u's errors, each weighed by
            z = x @ w.T                                  # at most 1.1 |u| (the slope's maximum) and |silu(g)|
            gate, up = z[:, :n], z[:, n:]
            want = mx.gated(gate, up, "silu")
            rms = np.linalg.norm(z) / np.sqrt(z.size) * limit(k, parts)
            allowed = rms * (1.1 * np.linalg.norm(up) + np.linalg.norm(mx.activation(gate, "silu")[0]))
            allowed += 2.0 ** -24 * (16 + 8 * np.abs(gate).max()) * np.linalg.norm(want)
            assert np.linalg.norm(f64(y) - want) <= allowed
        else:
            want = x @ w if kind == BACKWARD else x @ w.T
            error = relative_error(f64(y), want)
            report("mx_bf16_norm", tile=tile, kind=kind, parts=parts, error=f"{error:.2e}")
            assert error <= limit(n if kind == BACKWARD else k, parts)
