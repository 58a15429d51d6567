"""Products of bf16 rows with MXFP4 weights on the GPU, forward and backward, against
the fp64 oracle (oracle/mx.py).

Tolerances, from the arithmetic, with e = 2^-24:
* sums: each product is exact in fp32; adding T terms in any order, each addition
  rounded or cut to 24 bits, costs at most 2 T e of the sum of magnitudes.  Most
  shapes are tested on operands whose sums are exact whatever the order (small
  whole numbers times a power of two): these are compared bit for bit.
* a bf16 output is off by its rounding, 2^-9 of the value (half a step, 2^-8, over
  the binade's foot at most: 2^-8 is taken).
* act(g) * u, silu and gelu_tanh: the sigmoid is four roundings and two
  instructions of one unit in the last place, its argument's error (2^-24 of a
  polynomial of four operations, gelu_tanh) costs |z| of that: (16 + 8 |z|) e of the
  value; gelu: the complementary error function is good to 16 units in the last
  place, its argument's two roundings cost 2 x^2 <= g^2 each: (40 + 2 g^2) e.
  Values that involve numbers below 2^-126 may lose them: 2^-126 |g u| more.
* the slopes: the same for each of their two terms.
"""

import numpy as np
import pytest
import torch

from oracle import bits, mx
from tests.gpu_util import report

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
ACTS = ["silu", "gelu", "gelu_tanh"]
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def w4():
    import weight_only_bit_unpack_amd as m
    return m


def code(w4, act):
    return {"silu": w4.W4_SILU, "gelu": w4.W4_GELU, "gelu_tanh": w4.W4_GELU_TANH}[act]


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16(v):
    """fp64 -> the nearest bf16 values, as fp64."""
    return bits.bf16_to_f64(bits.rne_bf16(v))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(BF16).cuda()


def put(q):
    return torch.from_numpy(np.ascontiguousarray(q)).cuda()


def exact_weight(g, n, k):
    """Elements of 0.5 .. 6 and signs, scales 2^-1 .. 2^2: every product with a small
    whole number is a multiple of 2^-2, so sums stay exact up to 2^22."""
    c = g.integers(0, 16, (n, k)).astype(np.uint8)
    s = g.integers(126, 129, (n, k // 32)).astype(np.uint8)
    return put(mx.pack(c, "fp4")), put(s), mx.dequant(mx.pack(c, "fp4"), s, "fp4")


def exact_rows(g, m, k):
    return g.integers(-8, 9, (m, k)).astype(np.float64)


def weight(g, n, k, sigma=0.02):
    w = g.standard_normal((n, k)) * sigma * (0.5 + g.random((n, 1)))
    q, s = mx.quantize(w, "fp4")
    return put(q), put(s), mx.dequant(q, s, "fp4")


def canary(m, n, dtype, edge=256):
    """An [m, n] output of NaN inside a buffer whose edges must stay as they are."""
    buf = torch.full((m * n + 2 * edge,), 7.0, dtype=dtype, device="cuda")
    y = buf[edge:edge + m * n].view(m, n)
    y.fill_(float("nan"))
    return buf, y


def edges_kept(buf, m, n, edge=256):
    return bool((buf[:edge] == 7.0).all()) and bool((buf[edge + m * n:] == 7.0).all())


def same(y, want):
    """Equal to the exact sums, rounded once to y's type."""
    w = bf16(want) if y.dtype == BF16 else want
    got = f64(y)
    assert np.array_equal(got, w), np.argwhere(got != w)[:5]


def sums(y, want, bound, terms):
    got = f64(y)
    assert np.isfinite(got).all()
    tol = 2 * terms * E * bound
    if y.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    worst = np.max(np.abs(got - want) - tol)
    assert worst <= 0, worst


def act_tolerance(g, act):
    if act == "gelu":
        return (40 + 2 * g * g) * E
    z = g if act == "silu" else 1.6 * (g + 0.045 * g ** 3)
    return (16 + 8 * np.minimum(np.abs(z), 200)) * E


def gated_within(y, g, u, act):
    want = mx.gated(g, u, act)
    tol = act_tolerance(g, act) * np.abs(want) + 2.0 ** -126 * np.abs(g * u) + 2.0 ** -149
    if y.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    worst = np.max(np.abs(f64(y) - want) - tol)
    assert worst <= 0, worst


# m, n, k: single tokens, few rows, tiles and one beside, odd widths, short and long sums
SHAPES = [
    (1, 1, 32), (1, 64, 64), (1, 33, 96), (1, 2048, 2048), (1, 1000, 4128), (2, 257, 288), (3, 128, 256),
    (5, 130, 1056), (8, 96, 512), (9, 512, 2048), (13, 1023, 352), (15, 17, 160), (16, 256, 1024),
    (16, 31, 8192), (17, 64, 2080), (31, 129, 544), (32, 256, 2048), (33, 300, 96), (48, 128, 128),
    (64, 512, 4096), (65, 65, 1280), (100, 1000, 992), (127, 256, 5632), (128, 384, 224),
    (129, 127, 2048), (192, 130, 768), (256, 256, 1024), (257, 513, 2080), (300, 2048, 32), (511, 97, 4096),
    (700, 700, 672), (1024, 512, 1024), (1030, 1100, 1120), (40, 96, 384), (70, 300, 640), (600, 700, 2176),
    (2050, 1030, 160), (4100, 36, 96), (20, 9000, 64), (1, 7, 11008), (6, 8192, 64)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(w4, m, n, k):
    report("mx_linear_bf16", m=m, n=n, k=k)
    g = np.random.default_rng(m * 7 + n * 3 + k)
    wq, ws, w = exact_weight(g, n, k)
    x = exact_rows(g, m, k)
    for dtype in (F32, BF16):
        buf, y = canary(m, n, dtype)
        assert w4.w4_mx_linear_bf16(dev(x), wq, ws, y=y) is y
        same(y, x @ w.T)
        assert edges_kept(buf, m, n)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_grad(w4, m, n, k):
    report("mx_linear_grad", m=m, n=n, k=k)
    g = np.random.default_rng(m * 5 + n * 11 + k)
    wq, ws, w = exact_weight(g, n, k)
    dy = exact_rows(g, m, n)
    for dtype in (F32, BF16):
        buf, dx = canary(m, k, dtype)
        assert w4.w4_mx_linear_grad(dev(dy), wq, ws, dx=dx) is dx
        same(dx, dy @ w)
        assert edges_kept(buf, m, k)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated(w4, m, n, k, act):
    report("mx_gated_linear", m=m, n=n, k=k, act=act)
    g = np.random.default_rng(m * 3 + n * 5 + k)
    wq, ws, w = exact_weight(g, 2 * n, k)
    x = exact_rows(g, m, k) / 64 * 2.0 ** -int(np.log2(k) / 2)      # gates of a few units
    want = x @ w.T
    for dtype in (F32, BF16):
        buf, y = canary(m, n, dtype)
        gbuf, gu = canary(m, 2 * n, BF16)
        assert w4.w4_mx_gated_linear(dev(x), wq, ws, code(w4, act), gu=gu, y=y) is y
        same(gu, want)
        gated_within(y, want[:, :n], want[:, n:], act)
        assert edges_kept(buf, m, n) and edges_kept(gbuf, m, 2 * n)
        again = w4.w4_mx_gated_linear(dev(x), wq, ws, code(w4, act), y_dtype=dtype)
        assert torch.equal(again, y)                    # without gu, and the same bits every time


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated_grad(w4, m, n, k, act):
    report("mx_gated_linear_grad", m=m, n=n, k=k, act=act)
    g = np.random.default_rng(m + n * 7 + k * 3)
    wq, ws, w = weight(g, 2 * n, k)
    dh = dev(g.standard_normal((m, n)) * 1e-3)
    gu = dev(g.standard_normal((m, 2 * n)) * 2)
    gbuf, dgu = canary(m, 2 * n, BF16)
    buf, dx = canary(m, k, F32)
    out = w4.w4_mx_gated_linear_grad(dh, gu, wq, ws, code(w4, act), dgu=dgu, dx=dx)
    assert out[0] is dx and out[1] is dgu
    gate, up = f64(gu)[:, :n], f64(gu)[:, n:]
    dg, du = mx.gated_grad(f64(dh), gate, up, act)
    want = np.concatenate((dg, du), 1)
    a, d = mx.activation(gate, act)
    t = act_tolerance(gate, act) + 16 * E
    slope_terms = np.abs(d) + 2 * (1 + np.abs(gate))    # the terms that a slope is the sum of
    tol = np.concatenate((np.abs(f64(dh) * up) * slope_terms * t, np.abs(f64(dh) * a) * t), 1) + 2.0 ** -126
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(f64(dgu) - want) <= tol).all()
    s = f64(dgu)                                        # dx is of dgu as it is stored
    sums(dx, s @ w, np.abs(s) @ np.abs(w), 2 * n)
    assert edges_kept(buf, m, k) and edges_kept(gbuf, m, 2 * n)
    dx16, dgu16 = w4.w4_mx_gated_linear_grad(dh, gu, wq, ws, code(w4, act))
    assert dx16.dtype == BF16 and torch.equal(dgu16, dgu) and torch.equal(dx16, dx.to(BF16))
    over = gu.clone()                                   # dgu in gu's place
    dx2, dgu2 = w4.w4_mx_gated_linear_grad(dh, over, wq, ws, code(w4, act), dgu=over, dx_dtype=F32)
    assert dgu2 is over and torch.equal(over, dgu) and torch.equal(dx2, dx)


@pytest.mark.parametrize("m,n,k", [(1, 512, 2048), (7, 300, 1056), (40, 96, 4096), (300, 700, 2080), (1100, 513, 5632)])
def test_real_values(w4, m, n, k):
    """Normal weights and rows of very different size, both directions."""
    report("mx_bf16_real", m=m, n=n, k=k)
    g = np.random.default_rng(m + n + k)
    wq, ws, w = weight(g, n, k)
    x = dev(g.standard_normal((m, k)) * 10.0 ** g.uniform(-4, 4, (m, 1)))
    dy = dev(g.standard_normal((m, n)) * 10.0 ** g.uniform(-4, 4, (m, 1)))
    for dtype in (F32, BF16):
        sums(w4.w4_mx_linear_bf16(x, wq, ws, y_dtype=dtype), f64(x) @ w.T, np.abs(f64(x)) @ np.abs(w).T, k)
        sums(w4.w4_mx_linear_grad(dy, wq, ws, dx_dtype=dtype), f64(dy) @ w, np.abs(f64(dy)) @ np.abs(w), n)


@pytest.mark.parametrize("m", [1, 3, 16, 40, 130, 300])
def test_every_element_in_its_place(w4, m):
    """One nonzero per row against weights that tell every (row, k) apart."""
    report("mx_bf16_placement", m=m)
    n, k = 200, 1056
    g = np.random.default_rng(m)
    w = np.array([0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6])[g.integers(0, 14, (n, k))]
    w = w * 2.0 ** g.integers(-20, 20, (n, k // 32)).repeat(32, 1)
    q, s = mx.quantize(w, "fp4")
    w = mx.dequant(q, s, "fp4")
    x, dy = np.zeros((m, k)), np.zeros((m, n))
    at, to = g.integers(0, k, m), g.integers(0, n, m)
    x[np.arange(m), at] = 1.0
    dy[np.arange(m), to] = 1.0
    assert np.array_equal(f64(w4.w4_mx_linear_bf16(dev(x), put(q), put(s))), w.T[at])
    assert np.array_equal(f64(w4.w4_mx_linear_grad(dev(dy), put(q), put(s), dx_dtype=F32)), w[to])


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_every_scale_and_code(w4, m):
    """Each scale byte and element: the values that w4_mx_dequant gives as bf16, below
    2^-126 and above bf16's largest too, and NaN in the blocks of scale 255."""
    report("mx_bf16_scales", m=m)
    n, k = 256, 32
    q = mx.pack(np.resize(np.arange(16, dtype=np.uint8), (n, k)), "fp4")
    s = np.arange(256, dtype=np.uint8)[:, None]
    w = w4.w4_mx_dequant(put(q), put(s), w4.W4_MXFP4)
    wv = f64(w)
    for c in range(0, k, 3):
        x = np.zeros((m, k))
        x[:, c] = 1.0
        y = f64(w4.w4_mx_linear_bf16(dev(x), put(q), put(s)))
        # a NaN of the block reaches the sum, and so does 0 * infinity
        want = np.where(np.isfinite(wv).all(1), wv[:, c], np.nan)
        assert np.array_equal(y, np.tile(want, (m, 1)), equal_nan=True), c
    dy = np.zeros((m, n))
    rows = np.arange(m) * 7 % 200
    dy[np.arange(m), rows] = 1.0
    # (rows 253 .. 255 hold infinities and NaN)
    dx = f64(w4.w4_mx_linear_grad(dev(dy[:, :200].copy()), put(q[:200]), put(s[:200]), dx_dtype=F32))
    assert np.array_equal(dx, wv[rows])


@pytest.mark.parametrize("m", [2, 16, 60, 300])
def test_nan_and_infinity_stay_in_their_rows(w4, m):
    report("mx_bf16_nan", m=m)
    n, k = 96, 160                                       # sums that end inside a step
    g = np.random.default_rng(m)
    wq, ws, w = exact_weight(g, 2 * n, k)
    for bad in (np.nan, np.inf):
        x, dy = exact_rows(g, m, k), exact_rows(g, m, 2 * n)
        x[m - 1, k - 1] = dy[m - 1, 2 * n - 1] = bad
        for y, want in ((w4.w4_mx_linear_bf16(dev(x), wq, ws), x[:-1] @ w.T),
                        (w4.w4_mx_linear_grad(dev(dy), wq, ws, dx_dtype=F32), dy[:-1] @ w)):
            same(y[:-1], want)
            got = f64(y[-1])
            # infinity times an element of 0 is NaN
            assert (np.isnan(got) | np.isinf(got)).all() and (bad == np.inf or np.isnan(got).all())
        h = w4.w4_mx_gated_linear(dev(x), wq, ws)
        assert bool(torch.isfinite(h[:-1]).all())
    ws2 = ws.clone()
    ws2[3, k // 32 - 1] = 255
    x, dy = exact_rows(g, m, k), exact_rows(g, m, 2 * n)
    y = f64(w4.w4_mx_linear_bf16(dev(x), wq, ws2))
    assert np.isnan(y[:, 3]).all()
    keep = np.arange(2 * n) != 3
    assert np.array_equal(y[:, keep], (x @ w.T)[:, keep])
    y = f64(w4.w4_mx_linear_grad(dev(dy), wq, ws2, dx_dtype=F32))
    assert np.isnan(y[:, k - 32:]).all() and np.array_equal(y[:, :k - 32], (dy @ w)[:, :k - 32])


@pytest.mark.parametrize("act", ACTS)
def test_activation_over_its_range(w4, act):
    """Gates of every size of either sign, through one weight of value 1."""
    report("mx_gated_range", act=act)
    n, k = 64, 32
    q, s = np.zeros((2 * n, k // 2), np.uint8), np.full((2 * n, 1), 127, np.uint8)
    q[:n, 0], q[n:, 0] = 2, 2 << 4                       # gate rows take x[0], up rows x[1]
    mag = np.concatenate((np.linspace(0, 20, 801), np.geomspace(1e-30, 1e30, 400), np.linspace(80, 110, 200)))
    g = bf16(np.concatenate((mag, -mag)))
    x = np.zeros((len(g), k))
    x[:, 0], x[:, 1] = g, 1.5
    gu = torch.empty((len(g), 2 * n), dtype=BF16, device="cuda")
    y = w4.w4_mx_gated_linear(dev(x), put(q), put(s), code(w4, act), gu=gu)
    gate, up = np.tile(g[:, None], n), np.full((len(g), n), 1.5)
    assert np.array_equal(f64(gu), np.concatenate((gate, up), 1))
    gated_within(y, gate, up, act)
    _, dgu = w4.w4_mx_gated_linear_grad(dev(np.ones((len(g), n))), gu, put(q), put(s), code(w4, act))
    a, d = mx.activation(gate, act)
    t = np.minimum(act_tolerance(gate, act) + 16 * E, 1.0)
    tol = 1.5 * (np.abs(d) + 2 * np.minimum(1 + np.abs(gate), 40)) * t + 2.0 ** -126 * (1 + np.abs(gate))
    assert (np.abs(f64(dgu)[:, :n] - 1.5 * d) <= tol + 2.0 ** -8 * (np.abs(1.5 * d) + tol)).all()
    tol = np.abs(a) * t + 2.0 ** -126 * (1 + np.abs(gate))
    assert (np.abs(f64(dgu)[:, n:] - a) <= tol + 2.0 ** -8 * (np.abs(a) + tol)).all()
    # what is no number stays none
    x[:, 0] = np.nan
    assert bool(torch.isnan(w4.w4_mx_gated_linear(dev(x), put(q), put(s), code(w4, act))).all())


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(w4, act):
    """sum(dh * y) as a function of x, by central differences of the fp64 block with
    the rebuilt weights, against the two backward calls."""
    report("mx_gated_differences", act=act)
    m, n, k = 5, 48, 96
    g = np.random.default_rng(4)
    wq, ws, w = weight(g, 2 * n, k, 0.2)
    x, dh = bf16(g.standard_normal((m, k))), bf16(g.standard_normal((m, n)))
    gu = torch.empty((m, 2 * n), dtype=BF16, device="cuda")
    w4.w4_mx_gated_linear(dev(x), wq, ws, code(w4, act), gu=gu)
    dx, _ = w4.w4_mx_gated_linear_grad(dev(dh), gu, wq, ws, code(w4, act), dx_dtype=F32)
    loss = lambda v: (mx.gated(v @ w[:n].T, v @ w[n:].T, act) * dh).sum(-1)
    num = np.empty((m, k))
    for c in range(k):
        d = np.zeros(k)
        d[c] = 1e-4
        num[:, c] = (loss(x + d) - loss(x - d)) / 2e-4
    # gu and dgu are rounded to bf16: 2^-8 of the terms, whose derivatives are at most 1.2 (1 + |u|) each
    bound = (np.abs(dh) * (1.2 * (1 + np.abs(x @ w[n:].T)) + 1.2 * np.abs(x @ w[:n].T))) @ (np.abs(w[:n]) + np.abs(w[n:]))
    assert (np.abs(f64(dx) - num) <= 3 * 2.0 ** -8 * bound + 1e-6).all()


def test_y_aligned_to_one_element(w4):
    """Outputs that start at any element, of odd and even widths, as does gu."""
    report("mx_bf16_alignment")
    g = np.random.default_rng(3)
    for m, n, k in ((1, 40, 64), (9, 41, 96), (70, 128, 160), (300, 257, 128)):
        wq, ws, w = exact_weight(g, 2 * n, k)
        x, dy = exact_rows(g, m, k), exact_rows(g, m, 2 * n)
        for dtype in (F32, BF16):
            for edge in (256, 257, 258, 259):
                buf, y = canary(m, 2 * n, dtype, edge)
                w4.w4_mx_linear_bf16(dev(x), wq, ws, y=y)
                same(y, x @ w.T)
                assert edges_kept(buf, m, 2 * n, edge)
                buf, dx = canary(m, k, dtype, edge)
                w4.w4_mx_linear_grad(dev(dy), wq, ws, dx=dx)
                same(dx, dy @ w)
                assert edges_kept(buf, m, k, edge)
                buf, y = canary(m, n, dtype, edge)
                gbuf, gu = canary(m, 2 * n, BF16, edge)
                w4.w4_mx_gated_linear(dev(x / 64), wq, ws, gu=gu, y=y)
                same(gu, x / 64 @ w.T)
                gated_within(y, (x / 64 @ w.T)[:, :n], (x / 64 @ w.T)[:, n:], "silu")
                assert edges_kept(buf, m, n, edge) and edges_kept(gbuf, m, 2 * n, edge)


def test_empty_sizes(w4):
    report("mx_bf16_empty")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    b = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")
    full = lambda *s: torch.full(s, 3.0, device="cuda")
    assert w4.w4_mx_linear_bf16(b(0, 64), u8(6, 32), u8(6, 2)).shape == (0, 6)
    assert w4.w4_mx_linear_bf16(b(4, 64), u8(0, 32), u8(0, 2)).shape == (4, 0)
    assert bool((w4.w4_mx_linear_bf16(b(4, 0), u8(6, 0), u8(6, 0), y=full(4, 6)) == 0).all())
    assert w4.w4_mx_gated_linear(b(0, 64), u8(6, 32), u8(6, 2)).shape == (0, 3)
    assert w4.w4_mx_gated_linear(b(4, 64), u8(0, 32), u8(0, 2)).shape == (4, 0)
    gu = full(4, 6).to(BF16)
    assert bool((w4.w4_mx_gated_linear(b(4, 0), u8(6, 0), u8(6, 0), gu=gu, y=full(4, 3)) == 0).all())
    assert bool((gu == 0).all())
    assert w4.w4_mx_linear_grad(b(0, 6), u8(6, 32), u8(6, 2)).shape == (0, 64)
    assert w4.w4_mx_linear_grad(b(4, 6), u8(6, 0), u8(6, 0)).shape == (4, 0)
    assert bool((w4.w4_mx_linear_grad(b(4, 0), u8(0, 32), u8(0, 2), dx=full(4, 64)) == 0).all())
    dx, dgu = w4.w4_mx_gated_linear_grad(b(4, 0), b(4, 0), u8(0, 32), u8(0, 2), dx=full(4, 64))
    assert bool((dx == 0).all()) and dgu.shape == (4, 0)
    gu = torch.randn(4, 6, device="cuda").to(BF16)
    dx, dgu = w4.w4_mx_gated_linear_grad(torch.ones(4, 3, device="cuda").to(BF16), gu, u8(6, 0), u8(6, 0))
    assert dx.shape == (4, 0) and bool((dgu != 0).any())  # dgu is there without columns, too
    dx, dgu = w4.w4_mx_gated_linear_grad(b(0, 3), b(0, 6), u8(6, 32), u8(6, 2))
    assert dx.shape == (0, 64) and dgu.shape == (0, 6)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 6, 7, 9, 10])
def test_padding_does_not_reach_the_sums(w4, n):
    """The rows that the call pads lie in memory where an earlier call left NaN."""
    report("mx_bf16_padding", n=n)
    g = np.random.default_rng(n)
    wq, ws, w = exact_weight(g, 2 * n, 64)
    m = 40
    nans = torch.full((2 * m, 101), float("nan"), dtype=BF16, device="cuda")
    w4.w4_mx_linear_grad(nans, *exact_weight(g, 101, 64)[:2])
    dh, gu = dev(g.standard_normal((m, n))), dev(g.standard_normal((m, 2 * n)))
    dx, dgu = w4.w4_mx_gated_linear_grad(dh, gu, wq, ws, w4.W4_GELU, dx_dtype=F32)
    assert bool(torch.isfinite(dx).all())
    limit = 2 * 2 * n * E * (np.abs(f64(dgu)) @ np.abs(w)) + 2.0 ** -149
    assert (np.abs(f64(dx) - f64(dgu) @ w) <= limit).all()
    w4.w4_mx_linear_grad(nans, *exact_weight(g, 101, 64)[:2])
    dy = exact_rows(g, m, n)
    same(w4.w4_mx_linear_grad(dev(dy), wq[:n], ws[:n], dx_dtype=F32), dy @ w[:n])


# ------------------------------------------------------------------ together, streams, graphs
def block(w4, x, dy, up, down, act, gu, stream=None):
    """A feed-forward block and its backward pass: (y, dx)."""
    h = w4.w4_mx_gated_linear(x, *up, act, gu=gu, y_dtype=BF16, stream=stream)
    y = w4.w4_mx_linear_bf16(h, *down, y_dtype=BF16, stream=stream)
    dh = w4.w4_mx_linear_grad(dy, *down, stream=stream)
    dx, _ = w4.w4_mx_gated_linear_grad(dh, gu, *up, act, stream=stream)
    return y, dx


@pytest.mark.parametrize("m,hidden,ffn", [(1, 256, 352), (30, 512, 1000), (300, 512, 1001)])
def test_block_together(w4, m, hidden, ffn):
    """Forward and backward of y = down(act(gate) * up) in fp64 with the rebuilt weights.
    Each stage is rounded to bf16, 2^-8 of its terms, and handed on."""
    report("mx_bf16_block", m=m, hidden=hidden, ffn=ffn)
    ffn32 = (ffn + 31) // 32 * 32                        # the down projection's k
    g = np.random.default_rng(m)
    up_q, up_s, up = weight(g, 2 * ffn32, hidden, 0.05)
    dn_q, dn_s, dn = weight(g, hidden, ffn32, 0.05)
    x, dy = bf16(g.standard_normal((m, hidden))), bf16(g.standard_normal((m, hidden)))
    gu = torch.empty((m, 2 * ffn32), dtype=BF16, device="cuda")
    y, dx = block(w4, dev(x), dev(dy), (up_q, up_s), (dn_q, dn_s), w4.W4_SILU, gu)
    gate, u = x @ up[:ffn32].T, x @ up[ffn32:].T
    h = mx.gated(gate, u, "silu")
    assert (np.abs(f64(y) - h @ dn.T) <= 2.0 ** -7 * (np.abs(h) @ np.abs(dn).T) + 2.0 ** -8 * np.abs(h @ dn.T)).all()
    dh = dy @ dn
    dg, du = mx.gated_grad(dh, gate, u, "silu")
    want = dg @ up[:ffn32] + du @ up[ffn32:]
    # each of dh, g, u, dgu is off by 2^-8 of itself, and the slopes are at most 1.2 of those
    t = (np.abs(dh) * 1.2 * ((1 + np.abs(gate)) * np.abs(u) + np.abs(gate)))
    assert (np.abs(f64(dx) - want) <= 2.0 ** -6 * (t @ (np.abs(up[:ffn32]) + np.abs(up[ffn32:])))).all()


@pytest.mark.parametrize("m,ffn", [(1, 352), (40, 352), (300, 1056)])
def test_other_stream_and_graph_replay(w4, m, ffn):
    """The block on a side stream, and captured once and replayed with new rows, with
    eager work between the replays, equals the eager block."""
    report("mx_bf16_graph", m=m, ffn=ffn)
    hidden = 512
    g = np.random.default_rng(m)
    up, dn = weight(g, 2 * ffn, hidden, 0.05)[:2], weight(g, hidden, ffn, 0.05)[:2]
    x, dy = (dev(g.standard_normal((m, hidden))) for _ in range(2))
    gu = torch.empty((m, 2 * ffn), dtype=BF16, device="cuda")
    want = block(w4, x, dy, up, dn, w4.W4_GELU, gu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = block(w4, x, dy, up, dn, w4.W4_GELU, gu, stream=side)   # also makes this stream's workspaces
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = block(w4, x, dy, up, dn, w4.W4_GELU, gu)
    for _ in range(4):
        x.copy_(dev(g.standard_normal((m, hidden))))
        dy.copy_(dev(g.standard_normal((m, hidden))))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        want = block(w4, x, dy, up, dn, w4.W4_GELU, gu)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(w4):
    """Calls that need workspaces, enqueued on two streams without waiting."""
    report("mx_bf16_two_streams")
    g = np.random.default_rng(2)
    m, n, k = 40, 1001, 512
    sets = []
    for _ in range(2):
        wq, ws, w = exact_weight(g, n, k)
        dy = exact_rows(g, m, n)
        sets.append((dev(dy), wq, ws, dy @ w, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (dy, wq, ws, _, stream) in enumerate(sets):
            outs[i].append(w4.w4_mx_linear_grad(dy, wq, ws, dx_dtype=F32, stream=stream))
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        for dx in outs[i]:
            same(dx, s[3])


# ------------------------------------------------------------------ large buffers
@pytest.mark.parametrize("m", [1, 40])
def test_w_beyond_4_gib(w4, m):
    """Weight rows whose bytes lie past 2^32, as outputs, as terms and as up rows."""
    report("mx_bf16_w_beyond_4_gib", m=m)
    n, k = 1_060_000, 8192                               # 4.34 GB of elements
    g = np.random.default_rng(7)
    wq = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda")
    rows = [0, 1_048_575, 1_048_576, 1_055_555, n - 1]
    q, s, w = exact_weight(g, len(rows), k)
    for i, r in enumerate(rows):
        wq[r], ws[r] = q[i], s[i]
    x = exact_rows(g, m, k)
    y = w4.w4_mx_linear_bf16(dev(x), wq, ws)
    same(y[:, rows].contiguous(), x @ w.T)
    assert int((y != 0).sum()) <= len(rows) * m
    gu = torch.empty((m, n), dtype=BF16, device="cuda")
    w4.w4_mx_gated_linear(dev(x), wq, ws, gu=gu)
    same(gu[:, rows].contiguous(), x @ w.T)
    dy = exact_rows(g, m, len(rows))
    full = torch.zeros((m, n), dtype=BF16, device="cuda")
    full[:, rows] = dev(dy)
    same(w4.w4_mx_linear_grad(full, wq, ws, dx_dtype=F32), dy @ w)


def test_rows_beyond_4_gib(w4):
    """Rows of x and of y whose bytes lie past 2^32."""
    report("mx_bf16_rows_beyond_4_gib")
    g = np.random.default_rng(8)
    m, n, k = 70_000, 32_768, 32                         # 4.6 GB of bf16 y, and dy
    wq, ws, w = exact_weight(g, n, k)
    pick = [0, 33_333, 65_535, 65_536, m - 1]
    x = torch.randint(-8, 9, (m, k), device="cuda").to(BF16)
    y = w4.w4_mx_linear_bf16(x, wq, ws, y_dtype=BF16)
    same(y[pick], f64(x[pick]) @ w.T)
    y.zero_()
    dy = exact_rows(g, len(pick), n)
    y[pick] = dev(dy)
    dx = w4.w4_mx_linear_grad(y, wq, ws, dx_dtype=F32)
    same(dx[pick], dy @ w)


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refusals(w4):
    report("mx_bf16_refusals")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    b = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")
    wq, ws = u8(8, 32), u8(8, 2)
    for call, match in (
            (lambda: w4.w4_mx_linear_bf16(b(4, 64).half(), wq, ws), "x has dtype"),
            (lambda: w4.w4_mx_linear_bf16(b(4, 96), wq, ws), "x has shape"),
            (lambda: w4.w4_mx_linear_bf16(b(64, 4).t(), wq, ws), "contiguous"),
            (lambda: w4.w4_mx_linear_bf16(b(4, 64), wq, u8(8, 1)), "ws has shape"),
            (lambda: w4.w4_mx_linear_bf16(b(4, 64), wq, ws, y_dtype=torch.float16), "y_dtype"),
            (lambda: w4.w4_mx_linear_bf16(b(4, 64), wq, ws, y=torch.zeros(4, 9, device="cuda")), "y has shape"),
            (lambda: w4.w4_mx_linear_bf16(b(4, 64).cpu(), wq, ws), "must be a CUDA"),
            (lambda: w4.w4_mx_linear_bf16(None, wq, ws), "x is required"),
            (lambda: w4.w4_mx_gated_linear(b(4, 64), u8(7, 32), u8(7, 2)), "as many gate as up"),
            (lambda: w4.w4_mx_gated_linear(b(4, 64), wq, ws, gu=b(4, 4)), "gu has shape"),
            (lambda: w4.w4_mx_gated_linear(b(4, 64), wq, ws, gu=b(4, 8).half()), "gu has dtype"),
            (lambda: w4.w4_mx_linear_grad(b(4, 9), wq, ws), "dy has shape"),
            (lambda: w4.w4_mx_linear_grad(b(4, 8), wq, ws, dx_dtype=torch.float16), "dx_dtype"),
            (lambda: w4.w4_mx_linear_grad(b(4, 8), wq, ws, dx=b(4, 8)), "dx has shape"),
            (lambda: w4.w4_mx_gated_linear_grad(b(4, 8), b(4, 8), wq, ws), "dh has shape"),
            (lambda: w4.w4_mx_gated_linear_grad(b(4, 4), b(5, 8), wq, ws), "gu has shape"),
            (lambda: w4.w4_mx_gated_linear_grad(b(4, 4), b(4, 8), wq, ws, dgu=b(4, 4)), "dgu has shape")):
        with pytest.raises(ValueError, match=match):
            call()
    for act in (-1, 3):
        with pytest.raises(w4.W4Error):
            w4.w4_mx_gated_linear(b(4, 64), wq, ws, act)
        with pytest.raises(w4.W4Error):
            w4.w4_mx_gated_linear_grad(b(4, 4), b(4, 8), wq, ws, act)
    with pytest.raises(w4.W4Error):                      # x from an odd element on
        w4.w4_mx_linear_bf16(b(4 * 64 + 1)[1:].view(4, 64), wq, ws)


def test_activation_codes_that_are_none(w4):
    report("mx_bf16_activation_codes")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    b = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")
    wq, ws = u8(8, 32), u8(8, 2)
    for act, error in ((2 ** 32, w4.W4Error), (-2 ** 32 + 1, w4.W4Error), (2 ** 70, OverflowError),
                       ("silu", TypeError), (None, TypeError)):
        with pytest.raises(error):
            w4.w4_mx_gated_linear(b(4, 64), wq, ws, act)
        with pytest.raises(error):
            w4.w4_mx_gated_linear_grad(b(4, 4), b(4, 8), wq, ws, act)


# ------------------------------------------------------------------ shared memory
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (40, 1000, 256), (40, 1002, 256), (70, 1001, 256), (5, 3, 64),
                                   (300, 4104, 96)])
def test_dgu_over_gu(w4, m, n, k):
    """dgu may be gu's own memory."""
    report("mx_bf16_dgu_over_gu", m=m, n=n, k=k)
    g = np.random.default_rng(m + n)
    wq, ws = weight(g, 2 * n, k)[:2]
    dh, gu = dev(g.standard_normal((m, n))), dev(g.standard_normal((m, 2 * n)))
    dx, dgu = w4.w4_mx_gated_linear_grad(dh, gu, wq, ws, w4.W4_GELU)
    dx2, dgu2 = w4.w4_mx_gated_linear_grad(dh, gu, wq, ws, w4.W4_GELU, dgu=gu)
    assert dgu2.data_ptr() == gu.data_ptr()
    assert torch.equal(dgu, gu) and torch.equal(dx, dx2)


def test_two_graphs_of_one_stream(w4):
    """Two captured calls share their stream's workspace and counters; replayed by turns,
    with eager work on other streams between, both stay right."""
    report("mx_bf16_two_graphs")
    g = np.random.default_rng(5)
    side = torch.cuda.Stream()
    sets = []
    for m, n, k in ((40, 1001, 512), (96, 2048, 640)):
        wq, ws, w = exact_weight(g, n, k)
        sets.append([dev(exact_rows(g, m, n)), wq, ws, w])
    torch.cuda.synchronize()
    for dy, wq, ws, _ in sets:                            # makes the workspaces
        w4.w4_mx_linear_grad(dy, wq, ws, dx_dtype=F32, stream=side)
    torch.cuda.synchronize()
    graphs = []
    for dy, wq, ws, w in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            dx = w4.w4_mx_linear_grad(dy, wq, ws, dx_dtype=F32)
        graphs.append((graph, dx, dy, wq, ws, w))
    for i in range(6):
        for graph, dx, dy, wq, ws, w in graphs:
            rows = exact_rows(g, *dy.shape)
            dy.copy_(dev(rows))
            graph.replay()
            eager = w4.w4_mx_linear_grad(dy, wq, ws, dx_dtype=F32)
            torch.cuda.synchronize()
            same(dx, rows @ w)
            same(eager, rows @ w)


def test_two_threads(w4):
    """Calls of two host threads, each on a stream of its own, while both make their
    streams' first workspaces."""
    report("mx_bf16_two_threads")
    import threading
    g = np.random.default_rng(6)
    sets = []
    for m, n, k in ((40, 1001, 512), (64, 700, 1024)):
        wq, ws, w = exact_weight(g, n, k)
        dy = exact_rows(g, m, n)
        sets.append((dev(dy), wq, ws, dy @ w, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]

    def work(i):
        dy, wq, ws, _, stream = sets[i]
        for _ in range(30):
            outs[i].append(w4.w4_mx_linear_grad(dy, wq, ws, dx_dtype=F32, stream=stream))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i, s in enumerate(sets):
        assert len(outs[i]) == 30
        for dx in outs[i]:
            same(dx, s[3])
