"""MX operators on the GPU at the ends of their ranges, against the fp64 oracle
(oracle/mx.py).

Tolerance of the norm, from the arithmetic: the squares add up in fp64 and the
row's factor is a power of two, applied exactly, times a number that is rounded
to fp32 once; a value then takes two fp32 roundings, the factor's product and
gamma's.  So v = v_exact (1 + d), |d| <= tau = 4 * 2^-24, wherever v is a normal
fp32 number, and codes are those of some number in [v (1 - tau), v (1 + tau)].
"""

import numpy as np
import pytest
import torch

from oracle import mx
from tests.gpu_util import report
from tests.test_gpu_mx import FMTS, _chain, _chain_inputs, check_codes, code, dev, f64, rounded

pytestmark = pytest.mark.gpu

TAU = 4 * 2.0 ** -24


@pytest.fixture(scope="module")
def w4():
    import weight_only_bit_unpack_amd as m
    return m


# ------------------------------------------------------------------ RMS norm
def norm_matches(w4, x, gamma, eps, fmt, dt, residual=None):
    t, gm = dev(x, dt), dev(gamma, dt)
    y = torch.full_like(t, float("nan"))
    r = None if residual is None else dev(residual, dt)
    q, s, _ = w4.w4_mx_rmsnorm(t, gm, eps, code(w4, fmt), residual=r, y=y)
    h = f64(t) if r is None else rounded((f64(t) + f64(r)).astype(np.float32).astype(np.float64), dt)
    v = mx.rmsnorm(h, f64(gm), eps)
    check_codes(q.cpu().numpy(), s.cpu().numpy(), v, TAU, fmt)
    a, b = rounded(v * (1 - TAU), dt), rounded(v * (1 + TAU), dt)
    got = f64(y)
    assert ((np.minimum(a, b) <= got) & (got <= np.maximum(a, b))).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [1e-40, 1e-25, 1e-19, 1e19, 1e25, 8e37])
def test_rmsnorm_large_and_small_rows(w4, size, fmt, dt):
    """Finite rows whose squares pass fp32's range on either side."""
    report("mx_rmsnorm_range", size=size, fmt=fmt, dt=dt)
    g = np.random.default_rng(3)
    for rows, k in ((3, 32), (5, 512), (2, 4128)):
        x = np.clip(g.standard_normal((rows, k)), -4, 4) * size
        gamma = 1 + 0.2 * g.standard_normal(k)
        norm_matches(w4, x, gamma, 0.0, fmt, dt)
        norm_matches(w4, x, gamma, 0.0, fmt, dt, residual=np.zeros_like(x))


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_one_large_value(w4, fmt):
    """One value far above the others: theirs are small, not zero."""
    report("mx_rmsnorm_one_large", fmt=fmt)
    g = np.random.default_rng(4)
    x = 1 + g.random((4, 512))
    x[[0, 1, 2], [0, 300, 511]] = 3e38, -1e30, 1e20
    norm_matches(w4, x, np.ones(512), 1e-6, fmt, "f32")


@pytest.mark.parametrize("fmt", FMTS)
def test_rmsnorm_gamma_and_row_of_opposite_size(w4, fmt):
    """h * gamma passes fp32's range on either side, the norm does not."""
    report("mx_rmsnorm_gamma_range", fmt=fmt)
    g = np.random.default_rng(5)
    x = g.standard_normal((3, 256))
    for size, scale in ((1e30, 1e12), (1e-30, 1e-12)):
        norm_matches(w4, x * size, scale * (1 + g.random(256)), 0.0, fmt, "f32")


# ------------------------------------------------------------------ streams
def stream_calls(w4):
    """Every operator with outputs of its own, and its inputs."""
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(64, 512, generator=g, device="cuda").bfloat16()
    gm = torch.ones(512, device="cuda").bfloat16()
    xq, xs = w4.w4_mx_quantize(x, w4.W4_MXFP8)
    wq, ws = w4.w4_mx_quantize(torch.randn(256, 512, generator=g, device="cuda"))
    off = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    wg, wgs = wq.view(2, 128, 256), ws.view(2, 128, 16)
    return [
        lambda **s: w4.w4_mx_quantize(x, w4.W4_MXFP8, **s),
        lambda **s: (w4.w4_mx_dequant(xq, xs, w4.W4_MXFP8, **s),),
        lambda **s: w4.w4_mx_rmsnorm(x, gm, residual=x, **s),
        lambda **s: (w4.w4_mx_linear(xq, xs, wq, ws, **s),),
        lambda **s: (w4.w4_mx_grouped_linear(xq, xs, wg, wgs, off, **s),)]


@pytest.mark.parametrize("op", range(5))
def test_stream_argument_allocates_on_that_stream(w4, op):
    """With stream= the outputs that the call makes are that stream's: a block just
    freed on the caller's stream, where queued work may still use it, is not taken."""
    report("mx_stream_outputs", op=op)
    call = stream_calls(w4)[op]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    mine = call()
    freed = {t.data_ptr() for t in mine}
    del mine                                         # back to the caller's stream's pool
    torch.cuda.synchronize()
    got = call(stream=side)
    assert not freed & {t.data_ptr() for t in got}
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("tokens", [1, 200])
def test_stream_argument_runs_there(w4, tokens):
    """The chain of calls given stream= equals the chain on the current stream, and
    waits for that stream's own work only."""
    report("mx_stream_argument", tokens=tokens)
    a = _chain_inputs(np.random.default_rng(tokens), tokens)
    _chain(w4, *a)
    torch.cuda.synchronize()
    want = [a[9].clone(), a[10].clone()]
    x, side = a[0].clone(), torch.cuda.Stream()
    for rep in range(3):
        a[0].zero_(), a[9].fill_(float("nan")), a[10].fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            a[0].copy_(x)                            # before the calls in the side stream's order
        _chain(w4, *a, stream=side)
        side.synchronize()
        assert torch.equal(a[9], want[0]) and torch.equal(a[10], want[1]), rep


# ------------------------------------------------------------------ more than a launch holds
def repeats(t, part):
    """Every whole run of part's length in t equals part, and so does what is left."""
    n = part.shape[0]
    whole = t.shape[0] // n
    runs = t[:whole * n].view((whole,) + tuple(part.shape))
    return all(bool((runs[i:i + 64] == part).all()) for i in range(0, whole, 64)) and \
        torch.equal(t[whole * n:], part[:t.shape[0] - whole * n])


@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm_more_rows_than_a_launch(w4, residual):
    report("mx_rmsnorm_rows", residual=residual)
    g = torch.Generator("cuda").manual_seed(2)
    base = torch.randn(4096, 32, generator=g, device="cuda").bfloat16()
    gm = torch.rand(32, generator=g, device="cuda").bfloat16()
    rows = 2 ** 24 + 1                               # 256 threads each: 2^32 and 256 more
    x = torch.empty((rows, 32), dtype=torch.bfloat16, device="cuda")
    x[:-1].view(-1, 4096, 32).copy_(base)
    x[-1] = base[0]
    y, yb = torch.zeros_like(x), torch.empty_like(base)
    r, rb = (x, base) if residual else (None, None)
    qb, sb, rob = w4.w4_mx_rmsnorm(base, gm, residual=rb, y=yb)
    q, s, ro = w4.w4_mx_rmsnorm(x, gm, residual=r, y=y)
    assert repeats(q, qb) and repeats(s, sb) and repeats(y, yb)
    assert not residual or repeats(ro, rob)
    del x, y, q, s, ro


def test_quantize_and_rebuild_more_than_a_launch(w4):
    report("mx_quantize_blocks")
    rows, k = 2 ** 23 + 1, 4096                      # 2^24 and 2 blocks of 2048 values
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of GPU memory")
    g = torch.Generator("cuda").manual_seed(3)
    base = torch.randn(4096, k, generator=g, device="cuda").bfloat16()
    x = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda")
    x[:-1].view(-1, 4096, k).copy_(base)
    x[-1] = base[0]
    qb, sb = w4.w4_mx_quantize(base)
    q, s = w4.w4_mx_quantize(x)
    assert repeats(q, qb) and repeats(s, sb)
    x.zero_()
    w4.w4_mx_dequant(q, s, out=x)
    assert repeats(x, w4.w4_mx_dequant(qb, sb))
    del x, q, s
    torch.cuda.empty_cache()
