"""The mixture-of-experts example (examples/mx_moe_layer.py) on the GPU.

Its output against the layer computed token by token in fp64 from the
dequantized weights and the activations that the example's own calls produce,
stage by stage.  Tolerance: the two grouped products are rounded to bf16
(2^-8 of each) and the output once more; the sum over four experts has
weights that add to 1, so an output is within 2^-8 * (sum p |y| + |out|) plus
the products' own 1e-3 of the sum of magnitudes.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import mx
from tests.gpu_util import report

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("mx_moe_layer", os.path.join(ROOT, "examples", "mx_moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens", [1, 13, 150])
def test_layer_token_by_token(example, tokens):
    report("mx_moe_layer", tokens=tokens)
    w4 = example.w4
    weights = example.random_layer(512, 352, 8, 3, seed=tokens)
    layer = example.MxMoeLayer(**weights)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x = torch.randn((tokens, 512), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((tokens, 512), generator=g, device="cuda").to(torch.bfloat16)
    y, ro = layer(x, r)
    assert torch.equal(ro, (x.float() + r.float()).to(torch.bfloat16))

    f64 = lambda t: t.double().cpu().numpy()
    deq = lambda q, s, fmt: np.stack([mx.dequant(a, b, fmt) for a, b in zip(q.cpu().numpy(), s.cpu().numpy())])
    gu, dn = deq(*layer.gate_up, "fp4"), deq(*layer.down, "fp4")
    h = torch.empty_like(x)
    q, s, _ = w4.w4_mx_rmsnorm(x, layer.gamma, layer.eps, residual=r, y=h)
    xa = mx.dequant(q.cpu().numpy(), s.cpu().numpy(), "fp8")
    p, rows, offsets, place = layer.route(h)
    # the quantized activations between the products, as the example makes them
    a = w4.w4_mx_grouped_linear(q, s, *layer.gate_up, offsets, rows=rows, y_dtype=torch.bfloat16)
    gate, up = a.float().chunk(2, -1)
    act = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
    q2, s2 = w4.w4_mx_quantize(act, w4.W4_MXFP8)
    mid = mx.dequant(q2.cpu().numpy(), s2.cpu().numpy(), "fp8")

    logits = h.float() @ layer.router.float().t()
    top = torch.topk(torch.softmax(logits, -1), 3, -1)[1].cpu().numpy()
    pn, pl = f64(p), place.cpu().numpy().reshape(tokens, 3)
    ends, rn = offsets.cpu().numpy(), rows.cpu().numpy()
    for t in range(tokens):
        out, tol = np.zeros(512), np.zeros(512)
        for c in range(3):
            e, row = top[t, c], pl[t, c]
            assert ends[e] <= row < ends[e + 1] and rn[row] == t
            want, bound = mx.linear(xa[t:t + 1], gu[e])
            assert (np.abs(f64(a[row]) - want[0]) <= 1e-3 * bound[0] + 1e-6 + 2.0 ** -8 * np.abs(want[0])).all()
            yc, b = mx.linear(mid[row:row + 1], dn[e])
            out += pn[t, c] * yc[0]
            tol += pn[t, c] * (1e-3 * b[0] + 1e-6 + 2.0 ** -8 * np.abs(yc[0]))
        assert (np.abs(f64(y[t]) - out) <= tol + 2.0 ** -8 * (np.abs(out) + tol)).all(), t


def test_layer_in_a_graph(example):
    """Captured once, replayed with new tokens whose routing differs, against eager calls."""
    report("mx_moe_graph")
    layer = example.MxMoeLayer(**example.random_layer(512, 352, 8, 3))
    x = torch.empty((20, 512), dtype=torch.bfloat16, device="cuda")
    r = torch.empty_like(x)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def fill():
        for t in (x, r):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(torch.bfloat16))

    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y, ro = layer(x, r)
    for _ in range(3):
        fill()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want, wro = layer(x, r)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(ro, wro)
