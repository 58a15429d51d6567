"""Two host threads that call on one stream at once, past the interpreter's lock (the
library's C calls through ctypes, which lets it go): each call's outputs are the bits
that it gives alone."""

import ctypes
import threading

import pytest
import torch

from tests.gpu_util import report

pytestmark = pytest.mark.gpu

CALLS = 40


@pytest.fixture(scope="module")
def w4():
    import weight_only_bit_unpack_amd as m
    return m


def operands(kind, seed):
    """The tensors of one thread's calls, and call(y, stream)."""
    import weight_only_bit_unpack_amd as m
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    lib, p = m._lib, lambda t: t.data_ptr()
    if kind in ("gemm", "gemm_noalloc", "gemv"):
        rows, n, k = (16, 4096, 4096) if kind == "gemv" else (64, 256, 4096)
        packed, scales = m.w4_quantize_pack(rand(n, k), m.W4_DYADIC)
        x, call = rand(rows, k), getattr(lib, "w4_" + kind)
        return (packed, scales, x), (rows, n), lambda y, s: call(
            m.W4_DYADIC, n, k, p(packed), p(scales), None, p(x), rows, p(y), m.W4_F32, s)
    if kind == "mx_linear":
        rows, n, k = 64, 256, 8192
        (wq, ws), (xq, xs) = m.w4_mx_quantize(rand(n, k), m.W4_MXFP4), m.w4_mx_quantize(rand(rows, k), m.W4_MXFP8)
        return (wq, ws, xq, xs), (rows, n), lambda y, s: lib.w4_mx_linear(
            m.W4_MXFP8, n, k, p(wq), p(ws), p(xq), p(xs), rows, p(y), m.W4_F32, s)
    rows, n, k = 40, 1001, 512
    gated = kind == "mx_gated_linear_grad"
    wq, ws = m.w4_mx_quantize(rand(2 * n if gated else n, k), m.W4_MXFP4)
    dy = rand(rows, n)
    if not gated:
        return (wq, ws, dy), (rows, k), lambda y, s: lib.w4_mx_linear_grad(
            n, k, p(wq), p(ws), p(dy), rows, p(y), m.W4_F32, s)
    gu, dgu = rand(rows, 2 * n), torch.empty((rows, 2 * n), dtype=torch.bfloat16, device="cuda")
    return (wq, ws, dy, gu, dgu), (rows, k), lambda y, s: lib.w4_mx_gated_linear_grad(
        m.W4_SILU, n, k, p(wq), p(ws), p(dy), p(gu), rows, p(dgu), p(y), m.W4_F32, s)


@pytest.mark.parametrize("kind", ["gemm", "gemm_noalloc", "gemv", "mx_linear", "mx_linear_grad",
                                  "mx_gated_linear_grad"])
def test_two_threads_on_one_stream(w4, kind):
    report("threads", kind=kind)
    stream = torch.cuda.current_stream().cuda_stream
    sets = [operands(kind, seed) for seed in (1, 2)]
    want, outs = [], []
    for _, shape, call in sets:
        y = torch.full(shape, float("nan"), device="cuda")
        assert call(y, stream) == 0
        want.append(y)
        outs.append([torch.full(shape, float("nan"), device="cuda") for _ in range(CALLS)])
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(y).all()) for y in want) and not torch.equal(want[0], want[1])
    start, status = threading.Barrier(2), [[], []]

    def work(i):
        start.wait()
        for y in outs[i]:
            status[i].append(sets[i][2](y, ctypes.c_void_p(stream)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert status[i] == [0] * CALLS
        for y in outs[i]:
            assert torch.equal(y, want[i])
