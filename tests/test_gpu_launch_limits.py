"""Codec calls on weights of more threads' work than one launch holds (2^32): a
base weight repeated, whose results have to repeat."""

import pytest
import torch

from tests.gpu_util import report
from tests.test_gpu_mx_ranges import repeats

pytestmark = pytest.mark.gpu

BASE = 4096


def base_weight(k):
    g = torch.Generator("cuda").manual_seed(4)
    return (torch.randn(BASE, k, generator=g, device="cuda") * 0.02).bfloat16()


def repeated(base, rows):
    t = torch.empty((rows,) + tuple(base.shape[1:]), dtype=base.dtype, device="cuda")
    whole = rows // BASE
    t[:whole * BASE].view((whole,) + tuple(base.shape)).copy_(base)
    t[whole * BASE:] = base[:rows - whole * BASE]
    return t


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_warm_fit():
    """2 groups of 32 a block of 256 threads: from 2^30 weights on."""
    import weight_only_bit_unpack_amd as w4
    need(8)
    k, rows = 4096, 2 ** 18 + 3
    report("launch_limit_warm_fit", rows=rows, k=k)
    base = base_weight(k)
    cb, pb = w4.w4_signmag8_fit_warm(base, 1)
    w = repeated(base, rows)
    c = torch.zeros((rows, k // 32, 8), dtype=torch.float16, device="cuda")
    c, p = w4.w4_signmag8_fit_warm(w, 1, codebook=c)
    assert repeats(p, pb) and repeats(c, cb)


def test_quantize_and_dequant():
    """Eight weights a thread: from 2^35 weights on."""
    import weight_only_bit_unpack_amd as w4
    need(100)
    k, rows = 8192, 2 ** 22 + 1
    report("launch_limit_quantize", rows=rows, k=k)
    base = base_weight(k)
    pb, sb = w4.w4_quantize_pack(base)
    w = repeated(base, rows)
    p, s = w4.w4_quantize_pack(w)
    assert repeats(p, pb) and repeats(s, sb)
    w.zero_()
    w4.w4_unpack_dequant(p, scales=s, out=w)
    assert repeats(w, w4.w4_unpack_dequant(pb, scales=sb))
    del w, p, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("codec", ["LUT16", "SIGNMAG8", "DYADIC5", "LUT16S"])
def test_side_tables_of_a_second_launch(codec):
    """Past 2^33 weights each part takes its own scales and codebook."""
    import weight_only_bit_unpack_amd as w4
    need(60)
    k, rows = 8192, 2 ** 20 + 1
    report("launch_limit_tables", codec=codec)
    base, code = base_weight(k), getattr(w4, "W4_" + codec)
    w = repeated(base, rows)
    if codec == "DYADIC5":
        g = torch.Generator("cuda").manual_seed(5)
        wd = torch.randint(3, 6, (BASE, k // 64), generator=g, device="cuda", dtype=torch.uint8)
        small, large = w4.w4_quantize_dyadic5(base, wd), w4.w4_quantize_dyadic5(w, repeated(wd, rows))
        (pb, cb, sb), (p, c, s) = small, large
        assert repeats(c, cb)
    else:
        if codec == "SIGNMAG8":
            sb = s = None
            cb = w4.w4_signmag8_fit(base, 1)
            c = w4.w4_signmag8_fit(w, 1)
            assert repeats(c, cb)
        else:
            sb, cb = w4.w4_lut16_fit(base, 1)
            s, c = w4.w4_lut16_fit(w, 1)
            assert repeats(s, sb) and repeats(c, cb)
            if codec == "LUT16S":
                cb = c = torch.linspace(-1, 1, 16, device="cuda").bfloat16()
        pb, _ = w4.w4_quantize_pack(base, code, scales=sb, codebook=cb)
        p, _ = w4.w4_quantize_pack(w, code, scales=s, codebook=c)
    assert repeats(p, pb)
    if codec == "LUT16S":
        assert repeats(w4.w4_lut16s_interleave(p, s), w4.w4_lut16s_interleave(pb, sb))
    want = w4.w4_unpack_dequant(pb, code, scales=sb, codebook=cb)
    out = w.view(want.dtype)
    out.zero_()
    w4.w4_unpack_dequant(p, code, scales=s, codebook=c, out=out)
    assert repeats(out, want)
    del w, out, p, s, c
    torch.cuda.empty_cache()
