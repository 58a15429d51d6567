"""MX operators on the GPU against the fp64 oracle (oracle/mx.py).

Tolerances, from the arithmetic:
* quantize and rebuild are exact: compared bit for bit.
* RMS norm: the row's factor comes from fp32 partial sums of at most
  ``k / 256 + 8`` squares a lane (relative error at most that many 2^-24, half
  of it after the root) and is rounded once; the value takes two more
  roundings.  So v = v_exact (1 + d), |d| <= tau = (k / 512 + 8) 2^-24, and an
  output rounded to fewer bits must be what rounding some number in
  [v (1 - tau), v (1 + tau)] gives.
* Products with fp4 activations: every product and every sum of one matrix
  instruction is exact, the fp32 accumulator rounds once for each of the k/64
  instructions and a few times where partial sums meet:
  (k / 64 + 40) 2^-24 of the sum of magnitudes.
* Products with fp8 activations: the matrix core aligns a few neighbouring
  products to the largest and drops bits about 2^-14 below it, so eight
  neighbours lose at most 8 * 2^-13 < 1e-3 of their magnitudes: the GEMV
  tolerance, 1e-3 of the sum of magnitudes + 1e-6.
* A bf16 output adds its own rounding, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

from oracle import bits, matmul, mx
from tests.gpu_util import report

pytestmark = pytest.mark.gpu

FMTS = ["fp4", "fp8"]
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def w4():
    import weight_only_bit_unpack_amd as m
    return m


def code(w4, fmt):
    return w4.W4_MXFP4 if fmt == "fp4" else w4.W4_MXFP8


def f64(t):
    return t.detach().double().cpu().numpy()


def rounded(v, dt):
    """fp64 -> the values of the type, to nearest even, as fp64."""
    if dt == "bf16":
        return bits.bf16_to_f64(bits.rne_bf16(v))
    return v.astype(np.float16 if dt == "f16" else np.float32).astype(np.float64)


def dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DT[dt]).cuda()


def mixed(g, rows, k):
    """Values of many magnitudes, with zeros, whole zero blocks and ties."""
    x = g.standard_normal((rows, k)) * 2.0 ** g.integers(-6, 6, (rows, k // 32)).repeat(32, 1)
    x[g.random((rows, k)) < 0.05] = 0.0
    x[g.random((rows, k)) < 0.02] = -0.0
    t = g.random((rows, k)) < 0.1
    x[t] = np.round(x[t] * 4) / 4
    z = g.random((rows, k // 32)) < 0.1
    x[z.repeat(32, 1)] = 0.0
    return x


# ------------------------------------------------------------------ quantize, rebuild
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 64), (3, 96), (7, 1056), (257, 320), (64, 4096)])
def test_quantize_and_rebuild_exact(w4, rows, k, fmt, dt):
    report("mx_quantize", rows=rows, k=k, fmt=fmt, dt=dt)
    g = np.random.default_rng(rows * k)
    x = dev(mixed(g, rows, k), dt)
    q, s = w4.w4_mx_quantize(x, code(w4, fmt))
    qo, so = mx.quantize(f64(x), fmt)
    assert np.array_equal(s.cpu().numpy(), so)
    assert np.array_equal(q.cpu().numpy(), qo)
    want = mx.dequant(qo, so, fmt)
    assert np.array_equal(f64(w4.w4_mx_dequant(q, s, code(w4, fmt), out_dtype=torch.float32)), want)
    assert np.array_equal(f64(w4.w4_mx_dequant(q, s, code(w4, fmt))), rounded(want, "bf16"))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_every_bf16_value(w4, fmt):
    """Every finite bf16 value beside block maxima of every binade (its own and larger)."""
    report("mx_quantize_bf16_sweep", fmt=fmt)
    v = bits.all_finite_bf16()
    v = np.resize(v, (len(v) + 30) // 31 * 31).reshape(-1, 31)
    x = np.zeros((len(v), 32), dtype=np.uint16)
    x[:, :31] = v
    own = np.max(v & np.uint16(0x7FFF), axis=1)
    for up in (0, 0x80, 0x180, 0x300, 0x500):        # the block's maximum 0 .. 10 binades up
        x[:, 31] = np.minimum(own.astype(np.int64) + up, 0x7F7F).astype(np.uint16)
        t = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).cuda()
        q, s = w4.w4_mx_quantize(t, code(w4, fmt))
        qo, so = mx.quantize(bits.bf16_to_f64(x), fmt)
        assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo), up


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_fp32_extremes(w4, fmt):
    report("mx_quantize_fp32_extremes", fmt=fmt)
    tiny, big = np.float32(2.0 ** -149), np.finfo(np.float32).max
    rows = [np.zeros(32), np.full(32, -0.0), np.full(32, tiny), np.linspace(0, 1, 32) * 2.0 ** -126,
            np.linspace(-1, 1, 32) * big, np.full(32, big), np.where(np.arange(32) == 5, big, tiny),
            np.where(np.arange(32) == 5, 2.0 ** -120, tiny), np.linspace(0.9, 1.1, 32),
            np.where(np.arange(32) == 31, 1.0, 2.0 ** -np.arange(32.0))]
    x = np.array(rows, dtype=np.float32)
    t = torch.from_numpy(x).cuda()
    q, s = w4.w4_mx_quantize(t, code(w4, fmt))
    qo, so = mx.quantize(x.astype(np.float64), fmt)
    assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_non_finite(w4, fmt, dt):
    """A NaN or an infinity takes its own block and no other."""
    report("mx_quantize_non_finite", fmt=fmt, dt=dt)
    g = np.random.default_rng(2)
    x = g.standard_normal((6, 128))
    for i, (r, c) in enumerate([(0, 0), (1, 37), (2, 127), (3, 64), (4, 95)]):
        x[r, c] = (np.nan, np.inf, -np.inf)[i % 3]
    x[5, 32:64] = np.nan
    t = dev(x, dt)
    q, s = w4.w4_mx_quantize(t, code(w4, fmt))
    qo, so = mx.quantize(f64(t), fmt)
    assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo)
    v = f64(w4.w4_mx_dequant(q, s, code(w4, fmt)))
    assert np.array_equal(np.isnan(v), np.repeat(so == 255, 32, -1))


@pytest.mark.parametrize("fmt", FMTS)
def test_rebuild_every_code_and_scale(w4, fmt):
    report("mx_dequant_sweep", fmt=fmt)
    n = 16 if fmt == "fp4" else 256
    c = np.resize(np.arange(n, dtype=np.uint8), (256, max(n, 32)))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], c.shape[1] // 32, 1)
    q = mx.pack(c, fmt)
    want = mx.dequant(q, s, fmt)
    got = w4.w4_mx_dequant(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), code(w4, fmt),
                           out_dtype=torch.float32)
    with np.errstate(over="ignore"):
        assert np.array_equal(f64(got), want.astype(np.float32).astype(np.float64), equal_nan=True)
    got = w4.w4_mx_dequant(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), code(w4, fmt))
    fin = np.isfinite(want)
    assert np.array_equal(f64(got)[fin], rounded(want[fin], "bf16"))
    assert np.isnan(f64(got)[np.isnan(want)]).all()


# ------------------------------------------------------------------ RMS norm
def check_codes(q, s, v, tau, fmt):
    """Element codes and scales of some number within tau of each v."""
    lo, hi = v * (1 - tau), v * (1 + tau)
    s_lo, s_hi = mx.block_scales(lo, fmt), mx.block_scales(hi, fmt)
    assert ((s == s_lo) | (s == s_hi)).all()
    m = mx.SIGN[fmt] - 1
    c = mx.unpack(q, fmt)
    a, b = mx.codes(lo, s, fmt) & m, mx.codes(hi, s, fmt) & m
    assert ((np.minimum(a, b) <= (c & m)) & ((c & m) <= np.maximum(a, b))).all()
    assert ((c & ~np.uint8(m)) == np.where(np.signbit(v), mx.SIGN[fmt], 0))[(c & m) != 0].all()


NORM_SHAPES = [(1, 32), (1, 2048), (2, 96), (5, 1056), (33, 4096), (3, 5632), (2, 11008), (700, 256),
               (2, 16416), (1, 40000)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,k", NORM_SHAPES)
def test_rmsnorm(w4, rows, k, fmt, dt):
    report("mx_rmsnorm", rows=rows, k=k, fmt=fmt, dt=dt)
    g = np.random.default_rng(rows + k)
    x, r = dev(g.standard_normal((rows, k)), dt), dev(4 * g.standard_normal((rows, k)), dt)
    gm = dev(1 + 0.2 * g.standard_normal(k), dt)
    eps = float(np.float32(1e-5))
    tau = (k / 512 + 8) * 2.0 ** -24
    for residual in (None, r):
        y = torch.full_like(x, float("nan"))
        q, s, ro = w4.w4_mx_rmsnorm(x, gm, eps, code(w4, fmt), residual=residual, y=y)
        h = f64(x)
        if residual is None:
            assert ro is None
        else:
            h = rounded((h + f64(r)).astype(np.float32).astype(np.float64), dt)
            assert np.array_equal(f64(ro), h)
        v = mx.rmsnorm(h, f64(gm), eps)
        check_codes(q.cpu().numpy(), s.cpu().numpy(), v, tau, fmt)
        a, b = rounded(v * (1 - tau), dt), rounded(v * (1 + tau), dt)
        assert ((np.minimum(a, b) <= f64(y)) & (f64(y) <= np.maximum(a, b))).all()


def test_rmsnorm_in_place_and_norm_only(w4):
    report("mx_rmsnorm_in_place")
    g = np.random.default_rng(9)
    x, r = dev(g.standard_normal((19, 2048)), "bf16"), dev(g.standard_normal((19, 2048)), "bf16")
    gm = dev(1 + 0.1 * g.standard_normal(2048), "bf16")
    y0 = torch.empty_like(x)
    q0, s0, r0 = w4.w4_mx_rmsnorm(x, gm, 1e-6, residual=r, y=y0)
    for out in ("residual", "x"):
        xc, rc = x.clone(), r.clone()
        o = rc if out == "residual" else xc
        q, s, ro = w4.w4_mx_rmsnorm(xc, gm, 1e-6, residual=rc, residual_out=o)
        assert ro is o
        assert torch.equal(q, q0) and torch.equal(s, s0) and torch.equal(ro, r0)
    y = torch.empty_like(x)
    q, s, ro = w4.w4_mx_rmsnorm(x, gm, 1e-6, None, residual=r, y=y)
    assert q is None and s is None
    assert torch.equal(y, y0) and torch.equal(ro, r0)
    xc = x.clone()
    w4.w4_mx_rmsnorm(xc, gm, 1e-6, None, y=xc)       # the norm in x's own place
    w4.w4_mx_rmsnorm(x, gm, 1e-6, None, y=y)
    assert torch.equal(xc, y)


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_zero_and_non_finite_rows(w4, fmt):
    report("mx_rmsnorm_special", fmt=fmt)
    g = np.random.default_rng(10)
    x = g.standard_normal((5, 512))
    x[1] = 0.0
    x[2, 100] = np.nan
    x[3, 511] = np.inf
    t, gm = dev(x, "bf16"), dev(np.ones(512), "bf16")
    q, s, _ = w4.w4_mx_rmsnorm(t, gm, 1e-6, code(w4, fmt))
    v = f64(w4.w4_mx_dequant(q, s, code(w4, fmt)))
    assert (v[1] == 0).all()
    assert np.isnan(v[2]).all()                      # the factor is NaN
    # the factor is 0: 0 * x is 0, 0 * inf NaN, which takes its block
    assert (v[3, :480] == 0).all() and np.isnan(v[3, 480:]).all()
    assert np.isfinite(v[[0, 4]]).all()
    # a zero row without eps: 0 * inf
    q, s, _ = w4.w4_mx_rmsnorm(t[1:2].contiguous(), gm, 0.0, code(w4, fmt))
    assert (s == 255).all()


# ------------------------------------------------------------------ products
def operand(g, rows, k, fmt, sigma=1.0):
    """A random MX operand (rows: int or shape): bytes and values."""
    shape = (rows,) if isinstance(rows, int) else rows
    x = g.standard_normal(shape + (k,)) * sigma * 2.0 ** g.integers(-3, 4, shape + (1,))
    if k >= 64:
        x[..., g.integers(0, k, k // 64)] *= 20.0
    q, s = mx.quantize(x, fmt)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), mx.dequant(q, s, fmt)


def within(y, want, bound, fmt, k):
    got = f64(y)
    assert np.isfinite(got).all()
    tol = (k / 64 + 40) * 2.0 ** -24 * bound if fmt == "fp4" else \
        matmul.REL_TOL * bound + matmul.ABS_TOL
    if y.dtype == torch.bfloat16:
        tol = tol + matmul.BF16_OUT_REL * (np.abs(want) + tol)
    worst = np.max(np.abs(got - want) - tol)
    assert worst <= 0, worst


def canary(m, n, dtype):
    """An [m, n] output of NaN inside a buffer whose edges must stay as they are."""
    buf = torch.full((m * n + 512,), 7.0, dtype=dtype, device="cuda")
    y = buf[256:256 + m * n].view(m, n)
    y.fill_(float("nan"))
    return buf, y


def edges_kept(buf, m, n):
    return bool((buf[:256] == 7.0).all()) and bool((buf[256 + m * n:] == 7.0).all())


LINEAR = [  # m, n, k
    (1, 1, 32), (1, 64, 64), (1, 33, 96), (1, 2048, 2048), (1, 1000, 4128), (2, 257, 288), (3, 128, 256),
    (5, 130, 1056), (8, 96, 512), (9, 512, 2048), (13, 4095, 352), (15, 17, 160), (16, 256, 1024),
    (16, 31, 8192), (17, 64, 2080), (31, 129, 544), (32, 256, 2048), (33, 300, 96), (48, 128, 128),
    (64, 512, 4096), (65, 65, 1280), (100, 1000, 992), (127, 256, 5632), (128, 384, 224),
    (129, 127, 2048), (192, 130, 768), (256, 256, 1024), (257, 513, 2080), (300, 2048, 32), (511, 97, 4096),
    (700, 700, 672), (1024, 512, 1024), (1030, 1100, 1120),
    # rows of scales on whole dwords but no wider boundary
    (40, 96, 384), (70, 300, 640), (200, 257, 1152), (600, 700, 2176)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(w4, m, n, k, fmt, dtype):
    report("mx_linear", m=m, n=n, k=k, fmt=fmt, dtype=dtype)
    g = np.random.default_rng(m * 7 + n * 3 + k)
    xq, xs, x = operand(g, m, k, fmt)
    wq, ws, w = operand(g, n, k, "fp4", 0.02)
    buf, y = canary(m, n, dtype)
    out = w4.w4_mx_linear(xq, xs, wq, ws, code(w4, fmt), y=y)
    assert out is y
    want, bound = mx.linear(x, w)
    within(y, want, bound, fmt, k)
    assert edges_kept(buf, m, n)
    again = w4.w4_mx_linear(xq, xs, wq, ws, code(w4, fmt), y_dtype=dtype)
    assert torch.equal(again, y)                    # the same bits every time


# around the step counts at which a product's loop changes: 256 of k a step, 16
# scales copied at a time, up to four steps in flight, and ends inside a step
STEPS_K = [256 * s + d for s in (1, 2, 3, 4, 5, 6, 7, 9) for d in (-32, 0, 32, 128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n", [(40, 96), (150, 700), (600, 1100), (1100, 4200), (2300, 2900)])
def test_linear_step_counts(w4, m, n, fmt):
    g = torch.Generator("cuda").manual_seed(m + n)
    for k in STEPS_K:
        report("mx_linear_steps", m=m, n=n, k=k, fmt=fmt)
        xq, xs = w4.w4_mx_quantize(torch.randn(m, k, generator=g, device="cuda"), code(w4, fmt))
        wq, ws = w4.w4_mx_quantize(torch.randn(n, k, generator=g, device="cuda") * 0.02, w4.W4_MXFP4)
        x = w4.w4_mx_dequant(xq, xs, code(w4, fmt), out_dtype=torch.float32).double()
        w = w4.w4_mx_dequant(wq, ws, w4.W4_MXFP4, out_dtype=torch.float32).double()
        y = w4.w4_mx_linear(xq, xs, wq, ws, code(w4, fmt))
        wt = w.t().contiguous()
        within(y, f64(x @ wt), f64(x.abs() @ wt.abs()), fmt, k)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 4, 16, 40, 130, 300])
def test_linear_every_element_in_its_place(w4, m, fmt):
    """One nonzero x value per row against weights that tell every (row, k) apart."""
    report("mx_linear_placement", m=m, fmt=fmt)
    n, k = 96, 1056
    g = np.random.default_rng(m)
    x = np.zeros((m, k))
    at = g.integers(0, k, m)
    x[np.arange(m), at] = 1.0
    wv = np.array([0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6])
    w = wv[g.integers(0, len(wv), (n, k))] * 2.0 ** g.integers(-20, 20, (n, k // 32)).repeat(32, 1)
    q, s = mx.quantize(x, fmt)
    wq, ws = mx.quantize(w, "fp4")
    y = w4.w4_mx_linear(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), torch.from_numpy(wq).cuda(),
                        torch.from_numpy(ws).cuda(), code(w4, fmt))
    assert np.array_equal(f64(y), mx.dequant(wq, ws, "fp4").T[at])


@pytest.mark.parametrize("m", [1, 16, 50, 200])
def test_linear_scale_range_and_nan(w4, m):
    """Scales at both ends of the range, and NaN blocks and codes: their rows and
    columns are NaN, the others untouched."""
    report("mx_linear_scales", m=m)
    n, k = 70, 672
    g = np.random.default_rng(m)
    for fmt in FMTS:
        xq, xs, x = operand(g, m, k, fmt)
        wq, ws, w = operand(g, n, k, "fp4")
        # x up by 2^100, w down by 2^100: the same products
        up = 100
        y = w4.w4_mx_linear(xq, xs + up, wq, ws - up, code(w4, fmt))
        want, bound = mx.linear(x, w)
        within(y, want, bound, fmt, k)
        ws2, xs2 = ws.clone(), xs.clone()
        ws2[3, k // 32 - 1] = 255
        xs2[m - 1, 0] = 255
        y = f64(w4.w4_mx_linear(xq, xs2, wq, ws2, code(w4, fmt)))
        bad = np.zeros((m, n), bool)
        bad[m - 1], bad[:, 3] = True, True
        assert np.array_equal(np.isnan(y), bad)
        if fmt == "fp8":
            xq2 = xq.clone()
            xq2[0, k - 1] = 0x7F
            y = f64(w4.w4_mx_linear(xq2, xs, wq, ws, code(w4, fmt)))
            bad[:] = False
            bad[0] = True
            assert np.array_equal(np.isnan(y), bad)
        # all scales 0: 2^-254 of anything is 0
        y = w4.w4_mx_linear(xq, torch.zeros_like(xs), wq, torch.zeros_like(ws), code(w4, fmt))
        assert bool((y == 0).all())


def test_linear_empty_sizes(w4):
    report("mx_linear_empty")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    assert w4.w4_mx_linear(u8(0, 64), u8(0, 2), u8(5, 32), u8(5, 2)).shape == (0, 5)
    assert w4.w4_mx_linear(u8(4, 64), u8(4, 2), u8(0, 32), u8(0, 2)).shape == (4, 0)
    y = torch.full((4, 5), 3.0, device="cuda")
    w4.w4_mx_linear(u8(4, 0), u8(4, 0), u8(5, 0), u8(5, 0), y=y)
    assert bool((y == 0).all())
    x = torch.zeros((0, 64), device="cuda")
    q, s = w4.w4_mx_quantize(x)
    assert q.shape == (0, 32) and s.shape == (0, 2)
    assert w4.w4_mx_dequant(q, s).shape == (0, 64)
    q, s, r = w4.w4_mx_rmsnorm(x, torch.ones(64, device="cuda"))
    assert q.shape == (0, 64) and r is None


# ------------------------------------------------------------------ grouped products
def counts_to_offsets(c):
    return np.concatenate(([0], np.cumsum(c))).astype(np.int32)


GROUPED = [  # tokens, n, k, rows of each expert, spare rows, gather
    (1, 64, 64, [1], 0, False),
    (1, 300, 2048, [1, 0, 1, 1, 0, 0, 1, 0], 0, True),
    (5, 128, 96, [0, 0, 5], 0, False),
    (7, 257, 352, [3, 1, 0, 2, 0, 1], 5, True),
    (24, 512, 2048, [3, 0, 16, 17, 1, 2, 30, 0, 27], 32, True),
    (40, 130, 1056, [0] * 8, 40, True),
    (64, 96, 544, [64] + [0] * 15, 0, False),
    (100, 200, 288, [33, 31, 0, 32, 4], 3, True),
    (129, 127, 160, [129, 1, 128, 127], 0, True),
    (300, 256, 1024, [0, 65, 64, 63, 200, 0, 1], 0, True),
    (513, 384, 672, [512, 0, 1], 0, False),
    (90, 65, 32, [1] * 70 + [0] * 30 + [2] * 20, 9, True),
    (64, 33, 64, [0, 1] * 150 + [2] * 57, 1, True),
    (700, 513, 1280, [257, 255, 256, 300, 10, 0, 90], 100, True)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_linear(w4, case, fmt, dtype):
    tokens, n, k, counts, spare, gather = GROUPED[case]
    report("mx_grouped", case=case, fmt=fmt, dtype=dtype)
    g = np.random.default_rng(case)
    rows = sum(counts) + spare
    tokens = tokens if gather else rows
    idx = g.integers(0, tokens, rows).astype(np.int32) if gather else None
    off = counts_to_offsets(counts)
    xq, xs, x = operand(g, tokens, k, fmt)
    wq, ws, w = operand(g, (len(counts), n), k, "fp4", 0.02)
    want, bound = mx.grouped_linear(x, w, off, idx)
    buf, y = canary(rows, n, dtype)
    t_idx = None if idx is None else torch.from_numpy(idx).cuda()
    w4.w4_mx_grouped_linear(xq, xs, wq, ws, torch.from_numpy(off).cuda(), code(w4, fmt), rows=t_idx, y=y)
    within(y, want, bound, fmt, k)
    assert bool((y[sum(counts):] == 0).all())
    assert edges_kept(buf, rows, n)
    again = w4.w4_mx_grouped_linear(xq, xs, wq, ws, torch.from_numpy(off).cuda(), code(w4, fmt), rows=t_idx,
                                    y_dtype=dtype)
    assert torch.equal(again, y)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_padded_and_unordered_inputs(w4, fmt):
    """Row indices outside x are rows of zeros, also where x holds NaN; offsets that
    decrease or pass the number of rows read as the nearest that does not."""
    report("mx_grouped_odd_inputs", fmt=fmt)
    g = np.random.default_rng(77)
    tokens, n, k, E, rows = 20, 96, 320, 5, 150
    xq, xs, x = operand(g, tokens, k, fmt)
    wq, ws, w = operand(g, (E, n), k, "fp4")
    idx = g.integers(0, tokens, rows).astype(np.int32)
    for v in (-1, tokens, 2 ** 31 - 1, -2 ** 31):
        idx[g.integers(0, rows, 6)] = v
    xs[0] = 255                                      # the row a clamped index would read
    x0 = x.copy()
    x0[0] = np.nan
    idx[:3] = 0, -1, 0
    for off in ([0, 10, 20, 30, 40, 150], [0, 70, 30, 90, 80, 140], [9, 10, 1000, 20, 2 ** 31 - 1, 5],
                [0, -5, -2 ** 31, 60, 60, 61], [0, 0, 0, 0, 0, 0]):
        off = np.array(off, dtype=np.int64).astype(np.int32)
        want, bound = mx.grouped_linear(x, w, off, idx)
        nan, _ = mx.grouped_linear(x0, w, off, idx)
        buf, y = canary(rows, n, torch.float32)
        w4.w4_mx_grouped_linear(xq, xs, wq, ws, torch.from_numpy(off).cuda(), code(w4, fmt),
                                rows=torch.from_numpy(idx).cuda(), y=y)
        assert np.array_equal(np.isnan(f64(y)), np.isnan(nan))
        y[torch.isnan(y)] = 0.0
        keep = ~np.isnan(nan)
        within(y, np.where(keep, want, 0.0), np.where(keep, bound, 1.0), fmt, k)
        assert edges_kept(buf, rows, n)


def test_grouped_no_experts_and_no_tokens(w4):
    report("mx_grouped_none")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = torch.full((4, 8), 3.0, device="cuda")
    w4.w4_mx_grouped_linear(u8(4, 64), u8(4, 2), u8(0, 8, 32), u8(0, 8, 2), off, y=y)
    assert bool((y == 0).all())
    y.fill_(3.0)
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    w4.w4_mx_grouped_linear(u8(0, 64), u8(0, 2), u8(2, 8, 32), u8(2, 8, 2), off, rows=idx, y=y)
    assert bool((y == 0).all())


def test_grouped_matches_one_expert_at_a_time(w4):
    """Each group's rows equal the plain product of that expert, to the tolerance,
    whatever its size and position among the others."""
    report("mx_grouped_vs_linear")
    g = np.random.default_rng(5)
    counts = [40, 0, 1, 16, 200, 3]
    n, k = 256, 2048
    xq, xs, x = operand(g, sum(counts), k, "fp4")
    wq, ws, w = operand(g, (len(counts), n), k, "fp4", 0.02)
    off = counts_to_offsets(counts)
    y = w4.w4_mx_grouped_linear(xq, xs, wq, ws, torch.from_numpy(off).cuda(), w4.W4_MXFP4)
    for e in range(len(counts)):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            one = w4.w4_mx_linear(xq[lo:hi].contiguous(), xs[lo:hi].contiguous(), wq[e], ws[e], w4.W4_MXFP4)
            _, bound = mx.linear(x[lo:hi], w[e])
            assert (np.abs(f64(one) - f64(y[lo:hi])) <= 2 * (k / 64 + 40) * 2.0 ** -24 * bound).all()


# ------------------------------------------------------------------ large buffers
def test_x_beyond_4_gib(w4):
    """Row indices whose bytes lie past 2^32 in x."""
    report("mx_x_beyond_4_gib")
    k, tokens = 8192, 530_000                        # 4.34 GB of fp8 elements
    g = np.random.default_rng(6)
    xq = torch.zeros((tokens, k), dtype=torch.uint8, device="cuda")
    xs = torch.full((tokens, k // 32), 127, dtype=torch.uint8, device="cuda")
    rows = [tokens - 1, 0, 524_289, tokens - 2]
    q, s, x = operand(g, len(rows), k, "fp8")
    for i, r in enumerate(rows):
        xq[r], xs[r] = q[i], s[i]
    wq, ws, w = operand(g, (1, 40), k, "fp4", 0.02)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    y = w4.w4_mx_grouped_linear(xq, xs, wq, ws, off, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    want, bound = mx.linear(x, w[0])
    within(y, want, bound, "fp8", k)
    del xq, xs


@pytest.mark.parametrize("m", [1, 40])
def test_w_beyond_4_gib(w4, m):
    """Weight rows whose bytes lie past 2^32, as one weight and as the last expert."""
    report("mx_w_beyond_4_gib", m=m)
    n, k = 1_060_000, 8192                           # 4.34 GB of fp4 elements
    g = np.random.default_rng(7)
    wq = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda")
    cols = [0, 1_048_575, 1_048_576, 1_055_555, n - 1]
    q, s, w = operand(g, len(cols), k, "fp4")
    for i, c in enumerate(cols):
        wq[c], ws[c] = q[i], s[i]
    xq, xs, x = operand(g, m, k, "fp4")
    want, bound = mx.linear(x, w)
    y = w4.w4_mx_linear(xq, xs, wq, ws, w4.W4_MXFP4)
    within(y[:, cols].contiguous(), want, bound, "fp4", k)
    assert int((y != 0).sum()) <= len(cols) * m
    off = torch.tensor([0, 0, m], dtype=torch.int32, device="cuda")
    y = w4.w4_mx_grouped_linear(xq, xs, wq.view(2, n // 2, k // 2), ws.view(2, n // 2, k // 32), off, w4.W4_MXFP4)
    far = [c - n // 2 for c in cols if c >= n // 2]
    within(y[:, far].contiguous(), want[:, len(cols) - len(far):], bound[:, len(cols) - len(far):], "fp4", k)
    del wq, ws, y


def test_y_and_arrays_beyond_4_gib(w4):
    """More than 2^32 bytes of y, of a quantize call's input and of its values."""
    report("mx_y_beyond_4_gib")
    g = np.random.default_rng(8)
    m, n, k = 70_000, 32_768, 32                     # 4.6 GB of bf16
    xq, xs, x = operand(g, m, k, "fp4")
    wq, ws, w = operand(g, n, k, "fp4")
    y = w4.w4_mx_linear(xq, xs, wq, ws, w4.W4_MXFP4, y_dtype=torch.bfloat16)
    pick = [0, 33_333, 65_535, 65_536, m - 1]
    want, bound = mx.linear(x[pick], w)
    within(y[pick], want, bound, "fp4", k)
    q, s = w4.w4_mx_quantize(y, w4.W4_MXFP4)
    qo, so = mx.quantize(f64(y[pick]), "fp4")
    assert np.array_equal(q[pick].cpu().numpy(), qo) and np.array_equal(s[pick].cpu().numpy(), so)
    v = w4.w4_mx_dequant(q, s, w4.W4_MXFP4, out=y)
    assert np.array_equal(f64(v[pick]), rounded(mx.dequant(qo, so, "fp4"), "bf16"))
    gm = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    tail = y[-1:].clone()
    q1, s1, _ = w4.w4_mx_rmsnorm(tail, gm)
    q, s, _ = w4.w4_mx_rmsnorm(y, gm)
    assert torch.equal(q[-1], q1[0]) and torch.equal(s[-1], s1[0])
    del y, q, s, v


# ------------------------------------------------------------------ streams, graphs
def _chain(w4, x, r, gm, wq, ws, off, idx, wq2, ws2, y1, y2, stream=None):
    q, s, ro = w4.w4_mx_rmsnorm(x, gm, residual=r, stream=stream)
    w4.w4_mx_grouped_linear(q, s, wq, ws, off, rows=idx, y=y1, stream=stream)
    q, s = w4.w4_mx_quantize(y1, w4.W4_MXFP8, stream=stream)
    w4.w4_mx_linear(q, s, wq2, ws2, y=y2, stream=stream)


def _chain_inputs(g, tokens):
    k, n, n2, E = 2048, 512, 2048, 6
    x, r = dev(g.standard_normal((tokens, k)), "bf16"), dev(g.standard_normal((tokens, k)), "bf16")
    gm = dev(1 + 0.1 * g.standard_normal(k), "bf16")
    wq, ws, _ = operand(g, (E, n), k, "fp4", 0.02)
    wq2, ws2, _ = operand(g, n2, n, "fp4", 0.02)
    rows = 2 * tokens
    off = torch.from_numpy(np.sort(g.integers(0, rows + 1, E + 1)).astype(np.int32)).cuda()
    idx = torch.from_numpy(g.integers(0, tokens, rows).astype(np.int32)).cuda()
    y1 = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    y2 = torch.empty((rows, n2), device="cuda")
    return [x, r, gm, wq, ws, off, idx, wq2, ws2, y1, y2]


@pytest.mark.parametrize("tokens", [1, 20, 200])
def test_other_stream_and_graph_replay(w4, tokens):
    """The chain norm -> grouped -> quantize -> linear on a side stream, and captured
    once and replayed with new inputs and new groups, equals the eager chain."""
    report("mx_graph", tokens=tokens)
    g = np.random.default_rng(tokens)
    a = _chain_inputs(g, tokens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _chain(w4, *a)                               # also makes this stream's workspaces
    side.synchronize()
    got = [a[9].clone(), a[10].clone()]
    a[9].fill_(float("nan")), a[10].fill_(float("nan"))
    _chain(w4, *a)
    torch.cuda.synchronize()
    assert torch.equal(got[0], a[9]) and torch.equal(got[1], a[10])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        _chain(w4, *a)
    for rep in range(3):
        b = _chain_inputs(g, tokens)
        for i in (0, 1, 5, 6):
            a[i].copy_(b[i])
        a[9].fill_(float("nan")), a[10].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [a[9].clone(), a[10].clone()]
        _chain(w4, *a)
        torch.cuda.synchronize()
        assert torch.equal(got[0], a[9]) and torch.equal(got[1], a[10]), rep


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refusals(w4):
    report("mx_refusals")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    x = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError, match="multiple of 32"):
        w4.w4_mx_quantize(torch.zeros((4, 48), device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        w4.w4_mx_quantize(torch.zeros((64, 4), device="cuda").t())
    with pytest.raises(ValueError, match="dtype"):
        w4.w4_mx_quantize(x.double())
    with pytest.raises(ValueError, match="unknown MX format"):
        w4.w4_mx_quantize(x, 2)
    with pytest.raises(ValueError, match="scales has shape"):
        w4.w4_mx_dequant(u8(4, 32), u8(4, 3))
    with pytest.raises(ValueError, match="out has dtype"):
        w4.w4_mx_dequant(u8(4, 32), u8(4, 2), out=torch.zeros((4, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="gamma has shape"):
        w4.w4_mx_rmsnorm(x, torch.ones(32, device="cuda"))
    with pytest.raises(ValueError, match="gamma has dtype"):
        w4.w4_mx_rmsnorm(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="without a residual"):
        w4.w4_mx_rmsnorm(x, torch.ones(64, device="cuda"), residual_out=x)
    with pytest.raises(ValueError, match="y is required"):
        w4.w4_mx_rmsnorm(x, torch.ones(64, device="cuda"), fmt=None)
    with pytest.raises(w4.W4Error):
        w4.w4_mx_rmsnorm(x, torch.ones(64, device="cuda"), eps=-1.0)
    with pytest.raises(ValueError, match="xq has shape"):
        w4.w4_mx_linear(u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2), w4.W4_MXFP8)
    with pytest.raises(ValueError, match="ws has shape"):
        w4.w4_mx_linear(u8(4, 64), u8(4, 2), u8(8, 32), u8(8, 1))
    with pytest.raises(ValueError, match="y_dtype"):
        w4.w4_mx_linear(u8(4, 64), u8(4, 2), u8(8, 32), u8(8, 2), y_dtype=torch.float16)
    with pytest.raises(ValueError, match="y has shape"):
        w4.w4_mx_linear(u8(4, 64), u8(4, 2), u8(8, 32), u8(8, 2), y=torch.zeros((4, 9), device="cuda"))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="offsets has shape"):
        w4.w4_mx_grouped_linear(u8(4, 64), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2), off)
    with pytest.raises(ValueError, match="offsets has dtype"):
        w4.w4_mx_grouped_linear(u8(4, 64), u8(4, 2), u8(3, 8, 32), u8(3, 8, 2), off.long())
    with pytest.raises(ValueError, match="rows has dtype"):
        w4.w4_mx_grouped_linear(u8(4, 64), u8(4, 2), u8(3, 8, 32), u8(3, 8, 2), off, rows=off.long())
    with pytest.raises(ValueError, match="must be a CUDA"):
        w4.w4_mx_linear(u8(4, 64).cpu(), u8(4, 2), u8(8, 32), u8(8, 2))
    y = torch.full((4, 8), 7.0, device="cuda")
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())
