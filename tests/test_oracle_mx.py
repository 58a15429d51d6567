"""Pins for oracle/mx.py (microscaled blocks) on the CPU.

* the element levels against the formats' bit fields, by exact fractions;
* quantize against a brute-force nearest level in exact rational arithmetic,
  with planted ties, block extremes and the scale's clamped ends;
* rebuild and pack / unpack round trips;
* the products' group rule against rows picked one at a time.
"""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx


def _level_fraction(fmt, c):
    m, bias = (1, 1) if fmt == "fp4" else (3, 7)
    e, f = c >> m, c & ((1 << m) - 1)
    return Fraction(f, 1 << m) * Fraction(2) ** (1 - bias) if e == 0 else \
        (1 + Fraction(f, 1 << m)) * Fraction(2) ** (e - bias)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_levels(fmt):
    lev = mx.levels(fmt)
    assert [Fraction(v) for v in lev] == [_level_fraction(fmt, c) for c in range(len(lev))]
    assert list(lev) == sorted(lev)
    assert lev[-1] == (6.0 if fmt == "fp4" else 448.0)
    assert 2.0 ** mx.EMAX[fmt] <= lev[-1] < 2.0 ** (mx.EMAX[fmt] + 1)


def _brute(x, fmt):
    """(scale byte, codes) of one block by exact rational arithmetic."""
    a = max(abs(Fraction(v)) for v in x)
    e = -10_000
    if a:
        e = 0
        while Fraction(2) ** (e + 1) <= a:
            e += 1
        while Fraction(2) ** e > a:
            e -= 1
    b = min(max(e - mx.EMAX[fmt] + 127, 0), 254)
    s = Fraction(2) ** (b - 127)
    out = []
    for v in x:
        d = [abs(abs(Fraction(v)) - s * _level_fraction(fmt, c)) for c in range(len(mx.levels(fmt)))]
        best = [c for c in range(len(d)) if d[c] == min(d)]
        c = best[0] if len(best) == 1 else [c for c in best if c % 2 == 0][0]
        out.append(c + (mx.SIGN[fmt] if np.signbit(v) else 0))
    return b, out


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_quantize_vs_exact_rationals(fmt):
    g = np.random.default_rng(1)
    lev = mx.levels(fmt)
    blocks = []
    for i in range(12):
        x = g.standard_normal(32) * 2.0 ** g.integers(-20, 20)
        top = np.abs(x).max()
        s = 2.0 ** (np.floor(np.log2(top)) - mx.EMAX[fmt])
        j = g.integers(0, len(lev) - 1, 8)
        x[:8] = np.minimum((lev[j] + lev[j + 1]) / 2 * s, top) * np.where(g.random(8) < 0.5, -1, 1)  # ties
        x[8] = lev[-1] * s
        x[9], x[10] = 0.0, -0.0
        blocks.append(x)
    blocks.append(np.zeros(32))
    blocks.append(np.full(32, 2.0 ** -149))       # the smallest fp32 number
    blocks.append(np.full(32, 2.0 ** -120) * g.random(32))
    blocks.append(np.full(32, 3.4e38) * g.random(32))
    x = np.array(blocks)
    q, s = mx.quantize(x, fmt)
    c = mx.unpack(q, fmt)
    for i, row in enumerate(x):
        b, want = _brute(row, fmt)
        assert s[i, 0] == b and list(c[i]) == want, (i, s[i, 0], b)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_non_finite_blocks_and_rebuild(fmt):
    x = np.ones((4, 64))
    x[0, 3], x[1, 40], x[2, 0] = np.nan, np.inf, -np.inf
    q, s = mx.quantize(x, fmt)
    assert s.tolist() == [[255, 127 - mx.EMAX[fmt]], [127 - mx.EMAX[fmt], 255],
                          [255, 127 - mx.EMAX[fmt]], [127 - mx.EMAX[fmt]] * 2]
    v = mx.dequant(q, s, fmt)
    assert np.array_equal(np.isnan(v), np.repeat(s == 255, 32, -1))
    assert (v[~np.isnan(v)] == 1.0).all()
    assert (mx.unpack(q, fmt)[np.isnan(v)] == 0).all()


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_every_code_round_trips(fmt):
    n = 16 if fmt == "fp4" else 256
    c = np.arange(n, dtype=np.uint8)
    c = np.tile(c, 2) if fmt == "fp4" else c
    q = mx.pack(c[None], fmt)
    assert np.array_equal(mx.unpack(q, fmt)[0], c)
    s = np.full((1, len(c) // 32), 130, dtype=np.uint8)
    v = mx.dequant(q, s, fmt)[0]
    lev = mx.levels(fmt)
    for code, val in zip(c, v):
        m = int(code) & (mx.SIGN[fmt] - 1)
        if m >= len(lev):
            assert np.isnan(val)
        else:
            assert val == (-1 if code >= mx.SIGN[fmt] else 1) * lev[m] * 8.0
            assert np.signbit(val) == (code >= mx.SIGN[fmt])


def test_grouped_rows_one_at_a_time():
    g = np.random.default_rng(3)
    x, w = g.standard_normal((9, 32)), g.standard_normal((4, 5, 32))
    idx = np.array([0, 8, 3, -1, 9, 3, 2, 7, 1, 1])
    for offsets in ([0, 2, 2, 6, 8], [0, 0, 0, 0, 0], [5, 3, 1, 99, 4], [0, 10, 10, 10, 10]):
        y, b = mx.grouped_linear(x, w, offsets, idx)
        at = 0
        owner = [-1] * len(idx)
        for e in range(4):
            end = min(max(offsets[e + 1], at), len(idx))
            for t in range(at, end):
                owner[t] = e
            at = end
        for t, i in enumerate(idx):
            if owner[t] < 0 or not 0 <= i < 9:
                assert (y[t] == 0).all()
            else:
                assert np.allclose(y[t], w[owner[t]] @ x[i], rtol=1e-12)
                assert (b[t] >= np.abs(y[t]) - 1e-12).all()


def test_rmsnorm_scale_free():
    g = np.random.default_rng(4)
    h, gm = g.standard_normal((3, 64)), g.standard_normal(64)
    v = mx.rmsnorm(h, gm, 0.0)
    assert np.allclose(mx.rmsnorm(1e3 * h, gm, 0.0), v, rtol=1e-12)
    assert np.allclose((v / gm) ** 2 @ np.ones(64), 64.0)
