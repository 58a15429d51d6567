"""stream= of the codec calls: outputs that a call makes belong to that stream."""

import pytest
import torch

from tests.gpu_util import report

pytestmark = pytest.mark.gpu


def calls(w4):
    """Every codec call that makes outputs, as (name, function of stream=)."""
    g = torch.Generator("cuda").manual_seed(1)
    w = (torch.randn(64, 512, generator=g, device="cuda") * 0.02).bfloat16()
    x = torch.randn(4, 512, generator=g, device="cuda").bfloat16()
    p, s = w4.w4_quantize_pack(w)
    sl, cl = w4.w4_lut16_fit(w, 2)
    m = dict(scales=s)
    one = lambda f: lambda **kw: (f(**kw),)
    return [
        ("quantize_pack", lambda **kw: w4.w4_quantize_pack(w, **kw)),
        ("quantize_pack_lut16", lambda **kw: w4.w4_quantize_pack(w, w4.W4_LUT16, scales=sl, codebook=cl, **kw)[:1]),
        ("unpack_dequant", one(lambda **kw: w4.w4_unpack_dequant(p, scales=s, **kw))),
        ("quantize_dyadic5", lambda **kw: w4.w4_quantize_dyadic5(w, **kw)),
        ("lut16_fit", lambda **kw: w4.w4_lut16_fit(w, 2, **kw)),
        ("signmag8_fit", one(lambda **kw: w4.w4_signmag8_fit(w, 2, **kw))),
        ("signmag8_fit_warm", lambda **kw: w4.w4_signmag8_fit_warm(w, 2, **kw)),
        ("lut16s_interleave", one(lambda **kw: w4.w4_lut16s_interleave(p, s, **kw))),
        ("gemv", one(lambda **kw: w4.w4_gemv(p, x, **m, **kw))),
        ("gemm", one(lambda **kw: w4.w4_gemm(p, x, **m, **kw))),
        ("gemm_noalloc", one(lambda **kw: w4.w4_gemm_noalloc(p, x, **m, **kw))),
        ("linear", one(lambda **kw: w4.w4_linear(p, x, y_dtype=torch.bfloat16, **m, **kw)))]


@pytest.mark.parametrize("i", range(12))
def test_outputs_are_the_given_streams(i):
    """A block just freed on the caller's stream, where queued work may still use it,
    is not taken."""
    import weight_only_bit_unpack_amd as w4
    name, call = calls(w4)[i]
    report("stream_outputs", call=name)
    side = torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    mine = call()
    freed = {t.data_ptr() for t in mine}
    del mine
    torch.cuda.synchronize()
    got = call(stream=side)
    assert not freed & {t.data_ptr() for t in got}
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
