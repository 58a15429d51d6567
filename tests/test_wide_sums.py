"""That the operands and limits of tests/wide_sums.py do tell sums of 24 bits from
shorter ones: on the CPU, with sums cut or rounded on purpose."""

import numpy as np
import pytest

from tests.wide_sums import cut_sums, limit, relative_error, rounded_sums, wide


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("m,n,k", [(5, 130, 1056), (40, 96, 384), (17, 64, 2080), (9, 512, 8192)])
def test_wide_operands(m, n, k, back):
    q, s, w, x = wide(np.random.default_rng(m + n + k), m, n, k, back)
    a, b = (x, w.T) if back else (x, w)
    want = a @ b.T
    for order in (np.arange(a.shape[1]), np.random.default_rng(1).permutation(a.shape[1])):
        parts = np.cumsum(a[:, None, order] * b[None, :, order], -1)
        assert np.abs(parts).max() < 2 ** 22                 # 24 bits at quanta of 2^-2
        assert np.abs(parts).max() >= 2 ** 21
        assert np.array_equal(parts * 4, np.rint(parts * 4))
    assert np.array_equal(cut_sums(a, b, 24, 32), want)
    for bits in (16, 20, 22):
        assert (cut_sums(a, b, bits, 32) != want).mean() > 0.1, bits


@pytest.mark.parametrize("terms", [512, 2080, 5632, 11008])
def test_limits(terms):
    """Sums rounded to 24 bits an instruction of 16 (or of 4) terms stay within the limit, to
    22 bits not."""
    g = np.random.default_rng(terms)
    x, w = g.standard_normal((30, terms)), g.standard_normal((40, terms))
    want = x @ w.T
    assert relative_error(rounded_sums(x, w, 24), want) <= limit(terms)
    assert relative_error(rounded_sums(x, w, 24, 4), want) <= limit(terms)
    assert relative_error(rounded_sums(x, w, 22, 4), want) > limit(terms)
    assert relative_error(cut_sums(x, w, 22, 16), want) > limit(terms)


@pytest.mark.parametrize("bits", [8, 16, 18])
def test_limits_of_parts(bits):
    """Parts kept in fewer bits do not pass."""
    g = np.random.default_rng(bits)
    terms, parts = 1024, 8
    x, w = g.standard_normal((30, terms)), g.standard_normal((40, terms))
    total = 0
    for p in range(parts):
        at = slice(p * terms // parts, (p + 1) * terms // parts)
        f, e = np.frexp(x[:, at] @ w[:, at].T)
        total = total + np.ldexp(np.rint(np.ldexp(f, bits)), e - bits)
    assert relative_error(total, x @ w.T) > limit(terms, parts)
