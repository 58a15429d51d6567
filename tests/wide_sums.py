"""Operands and limits that tell sums of 24 bits from shorter ones, for the products of
bf16 rows with MXFP4 weights (test_gpu_mx_bf16_precision.py; on the CPU,
test_wide_sums.py).

Wide operands: every product is a multiple of 2^-2, and each row of x holds a term of
2^21 that a later one cancels, so that a running sum between them is a number of 24
bits at quanta of 2^-2 and the sum in the end a small one.  All partial sums, in any
order, stay below 2^22 as long as the other terms' do below 2^20: a 24-bit sum is exact, one that
keeps fewer bits loses the small terms' last ones.

Limits on the 2-norm of fp32 outputs of normal data, relative to the result's:
u (2 + sqrt(T / 32 + P / 2)), u = 2^-24, for T terms in P parts.  An addition that
rounds to nearest is off by 0.42 u of its sum (the root mean square over a binade:
2^-23 / sqrt 12 on average over the mantissas), and sums of random terms grow as
sqrt t, so n additions are off by 0.42 u sqrt(n / 2) of the result together.  A matrix
instruction adds 16 products or more; were each four of them rounded into the sum, n = T / 4,
that is 0.15 u sqrt T; the limit takes 0.18.  P parts add P additions of their own, for
which u is taken, and the 2 holds the last roundings.
"""

import numpy as np

from oracle import mx

BIG = 2.0 ** 19                # of x, times 4
PAIRS = 8


def limit(terms, parts=1):
    return 2.0 ** -24 * (2 + np.sqrt(terms / 32 + parts / 2))


def relative_error(got, want):
    return np.linalg.norm(np.asarray(got, dtype=np.float64) - want) / np.linalg.norm(want)


def _pairs(g, terms):
    """Up to PAIRS pairs of terms, none twice: the first and last, neighbours, and any."""
    free = g.permutation(np.setdiff1d(np.arange(terms), [0, terms // 2 - 1, terms // 2, terms - 1]))
    pairs = [(0, terms - 1), (terms // 2 - 1, terms // 2)]
    return pairs + [tuple(sorted(free[2 * i:2 * i + 2])) for i in range(min(PAIRS - 2, len(free) // 2))]


def wide(g, m, n, k, back=False):
    """(element bytes, scales, W, x), all on the host: W [n, k], x [m, k] (back: [m, n]).
    The sum goes over W's columns, back over its rows."""
    c = g.integers(0, 16, (n, k)).astype(np.uint8)
    s = g.integers(126, 130, (n, k // 32)).astype(np.uint8)      # 2^-1 .. 2^2
    terms = n if back else k
    x = g.integers(-8, 9, (m, terms)).astype(np.float64)
    if terms >= 4:
        pairs = _pairs(g, terms)
        for a, b in pairs:                                       # +-4 at scale 1, alike in both
            sign = (8 * g.integers(0, 2, k if back else n)).astype(np.uint8)
            if back:
                c[a] = c[b] = 6 + sign
                s[a] = s[b] = 127
            else:
                c[:, a] = c[:, b] = 6 + sign
                s[:, a // 32] = s[:, b // 32] = 127
        for row in range(m):
            own = [pairs[row % len(pairs)]]
            for a, b in pairs + own:                             # the row's own pair last
                x[row, a] = x[row, b] = 0
            (a, b), big = own[0], BIG if row % 3 else -BIG
            x[row, a], x[row, b] = big, -big
    q = mx.pack(c, "fp4")
    return q, s, mx.dequant(q, s, "fp4"), x


def cut_sums(x, w, bits, step=64):
    """x @ w.T in steps of terms, the running sum cut to so many significant bits after
    each."""
    total = np.zeros((x.shape[0], w.shape[0]))
    for t in range(0, x.shape[1], step):
        total = total + x[:, t:t + step] @ w[:, t:t + step].T
        f, e = np.frexp(total)
        total = np.ldexp(np.trunc(np.ldexp(f, bits)), e - bits)
    return total


def rounded_sums(x, w, bits, step=16):
    """The same, rounded to the nearest."""
    total = np.zeros((x.shape[0], w.shape[0]))
    for t in range(0, x.shape[1], step):
        f, e = np.frexp(total + x[:, t:t + step] @ w[:, t:t + step].T)
        total = np.ldexp(np.rint(np.ldexp(f, bits)), e - bits)
    return total
