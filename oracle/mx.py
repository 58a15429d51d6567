"""MX (microscaled) blocks: quantize, rebuild, the RMS norm and the products.

Oracle (test infrastructure).  The forms are the OCP Microscaling Formats
specification's: blocks of 32 consecutive values share a power-of-two scale
byte (E8M0, ``2**(b - 127)``, 255 = NaN); the elements are E2M1 (``fp4``) or
E4M3 (``fp8``).  Written from the definition of the element formats as sorted
lists of levels, in fp64: a block's scale exponent is that of its largest
magnitude less the largest element's, and a value takes the nearest level of
the scaled grid, the even code on a tie, the largest level beyond the grid.

Pinned against exact rational arithmetic in ``tests/test_oracle_mx.py``; the
activations of the gated block against their definitions and differences in
``tests/test_oracle_mx_gated.py``.
"""

import math

import numpy as np

BLOCK = 32
EMAX = {"fp4": 2, "fp8": 8}
SIGN = {"fp4": 8, "fp8": 128}


def levels(fmt):
    """Non-negative element values by code (sign bit clear), in order."""
    if fmt == "fp4":  # 2 exponent bits, 1 mantissa bit, bias 1
        sub, bias, m, codes = 2, 1, 1, 8
    else:             # 4 exponent bits, 3 mantissa bits, bias 7; the last code is NaN
        sub, bias, m, codes = 8, 7, 3, 127
    out = []
    for c in range(codes):
        e, f = c >> m, c & (sub - 1)
        out.append(f * 2.0 ** (1 - bias - m) if e == 0 else (sub + f) * 2.0 ** (e - bias - m))
    return np.array(out)


def block_scales(x, fmt):
    """fp64 [..., k] -> scale bytes uint8 [..., k/32]."""
    b = np.abs(np.asarray(x, dtype=np.float64)).reshape(x.shape[:-1] + (-1, BLOCK))
    bad = ~np.isfinite(b).all(-1)
    a = np.where(np.isfinite(b), b, 0.0).max(-1, initial=0.0)
    _, e = np.frexp(a)                       # a in [2**(e-1), 2**e)
    s = np.clip(e.astype(np.int64) - 1 - EMAX[fmt] + 127, 0, 254)
    s = np.where(a == 0.0, 0, s)
    return np.where(bad, 255, s).astype(np.uint8)


def codes(x, scales, fmt):
    """Element codes (one per value) of fp64 [..., k] at the given scales."""
    lev = levels(fmt)
    x = np.asarray(x, dtype=np.float64)
    s = np.repeat(scales.astype(np.int64), BLOCK, -1)
    with np.errstate(invalid="ignore"):
        m = np.ldexp(np.abs(np.where(np.isfinite(x), x, 0.0)), 127 - s)  # exact in fp64's range
    mid = (lev[1:] + lev[:-1]) / 2
    lo = np.searchsorted(mid, m, side="left")          # the lower level of a tie
    tie = (lo < len(mid)) & (mid[np.minimum(lo, len(mid) - 1)] == m)
    c = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    c = c + np.where(np.signbit(x), SIGN[fmt], 0)
    return np.where(s == 255, 0, c).astype(np.uint8)


def pack(c, fmt):
    """Codes -> the element bytes (fp4: two per byte, the even one low)."""
    return c if fmt == "fp8" else (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(q, fmt):
    if fmt == "fp8":
        return q
    return np.stack((q & 15, q >> 4), -1).reshape(q.shape[:-1] + (2 * q.shape[-1],))


def quantize(x, fmt):
    """fp64 [..., k] -> (element bytes, scale bytes)."""
    s = block_scales(x, fmt)
    return pack(codes(x, s, fmt), fmt), s


def dequant(q, scales, fmt):
    """fp64 values [..., k]."""
    lev = levels(fmt)
    if fmt == "fp8":
        lev = np.append(lev, np.nan)
    table = np.concatenate((lev, -lev))
    v = np.ldexp(table[unpack(q, fmt)], np.repeat(scales.astype(np.int64), BLOCK, -1) - 127)
    return np.where(np.repeat(scales, BLOCK, -1) == 255, np.nan, v)


def rmsnorm(h, gamma, eps):
    """fp64 [rows, k]: h * gamma / sqrt(mean(h**2) + eps)."""
    h = np.asarray(h, dtype=np.float64)
    ms = (h * h).sum(-1, keepdims=True) / h.shape[-1]
    return h * np.asarray(gamma, dtype=np.float64) / np.sqrt(ms + eps)


def linear(x, w):
    """fp64 (y, bound): x [m, k] w [n, k]^T and the sum of the terms' magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def groups(offsets, rows):
    """The half-open row range of each expert: offsets read in order, none below
    the one before it or above the number of rows, the first one as 0."""
    out, at = [], 0
    for end in list(offsets)[1:]:
        end = min(max(int(end), at), rows)
        out.append((at, end))
        at = end
    return out


def grouped_linear(x, w, offsets, row_index=None, rows=None):
    """fp64 (y, bound) of the products grouped by expert: x [tokens, k], w
    [experts, n, k]; rows of no expert, and rows whose index is outside x, are
    zeros."""
    rows = len(row_index) if row_index is not None else (x.shape[0] if rows is None else rows)
    src = np.arange(rows) if row_index is None else np.asarray(row_index, dtype=np.int64)
    ok = (src >= 0) & (src < x.shape[0])
    xs = np.where(ok[:, None], x[np.where(ok, src, 0)], 0.0) if rows else np.zeros((0, x.shape[1]))
    y, b = np.zeros((rows, w.shape[1])), np.zeros((rows, w.shape[1]))
    for e, (lo, hi) in enumerate(groups(offsets, rows)):
        if hi > lo:
            y[lo:hi], b[lo:hi] = linear(xs[lo:hi], w[e])
            y[lo:hi][~ok[lo:hi]] = 0.0
    return y, b


# ------------------------------------------------------------------ the gated block
def _erfc(x):
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


def _sigmoid(z):
    """1 / (1 + e^-z) without overflow, for either sign."""
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


TANH_A = math.sqrt(2.0 / math.pi)


def activation(g, act):
    """fp64 (act(g), act'(g)) of silu, gelu and gelu_tanh."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        return g * _sigmoid(g), _sigmoid(g) * (1 + g * _sigmoid(-g))
    if act == "gelu":
        phi = 0.5 * _erfc(-g / math.sqrt(2.0))
        return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if act != "gelu_tanh":
        raise ValueError(act)
    z = 2 * TANH_A * (g + 0.044715 * g ** 3)          # (1 + tanh(z / 2)) / 2 = sigmoid(z)
    slope = 2 * TANH_A * (1 + 3 * 0.044715 * g * g)
    return g * _sigmoid(z), _sigmoid(z) * (1 + g * _sigmoid(-z) * slope)


def gated(g, u, act):
    """fp64 act(g) * u."""
    return activation(g, act)[0] * np.asarray(u, dtype=np.float64)


def gated_grad(dh, g, u, act):
    """fp64 gradients of g and u, given that of act(g) * u."""
    a, d = activation(g, act)
    return np.asarray(dh) * np.asarray(u) * d, np.asarray(dh) * a
