"""Workloads of the MX operators: quantize + rebuild, RMS norm, linear and grouped linear.

The MX forms are the OCP microscaling ones: blocks of 32 values along k share
one power-of-two scale (E8M0, 2**(b - 127), 255 = NaN); elements are E2M1
("fp4", two per byte, low nibble first) or E4M3 ("fp8").  ``run`` computes each
operator either in plain elementary torch operations in 32 bits (``own``
false) or through the package's entry points (``own`` true).
"""

import torch

own = False

BLOCK = 32
#: (largest exponent, mantissa bits, smallest exponent of a normal, largest value) of an element
GRID = {"fp4": (2, 1, 0, 6.0), "fp8": (8, 3, -6, 448.0)}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # loading a model: the 11008 x 4096 projection of a 3.9B-sized model to MXFP4, read back dense
        {"name": "quant_weight_fp4", "op": "quant", "rows": 11008, "k": 4096, "fmt": "fp4", "dtype": "bf16"},
        # activations of an odd batch between two layers, 65 blocks a row
        {"name": "quant_act_fp8", "op": "quant", "rows": 333, "k": 2080, "fmt": "fp8", "dtype": "f16"},
        # decode, one token of the 1B-sized model: latency only
        {"name": "norm_token", "op": "norm", "rows": 1, "k": 2048, "fmt": "fp8", "dtype": "bf16", "residual": True},
        # prefill of a 3.9B-sized model
        {"name": "norm_prefill", "op": "norm", "rows": 8192, "k": 4096, "fmt": "fp8", "dtype": "bf16", "residual": True},
        # decode, one token through a 4096 -> 11008 projection: weight traffic only
        {"name": "linear_token", "op": "linear", "m": 1, "n": 11008, "k": 4096, "fmt": "fp8", "y": "bf16"},
        # a decode batch of odd size through a down projection, 4-bit activations
        {"name": "linear_batch13", "op": "linear", "m": 13, "n": 4095, "k": 5632, "fmt": "fp4", "y": "f32"},
        # the prefill product of 256 tokens, 8192 x 8192
        {"name": "linear_256", "op": "linear", "m": 256, "n": 8192, "k": 8192, "fmt": "fp8", "y": "bf16"},
        # a long prompt, 4-bit activations: matrix-core bound
        {"name": "linear_prompt", "op": "linear", "m": 4096, "n": 11008, "k": 4096, "fmt": "fp4", "y": "f32"},
        # one decoded token through 4 of 32 experts (gate and up projections side by side)
        {"name": "grouped_token", "op": "grouped", "tokens": 1, "rows": 4, "used": 4, "experts": 32, "active": 4,
         "n": 4096, "k": 2048, "fmt": "fp8", "y": "bf16", "gather": True},
        # a decode batch of 24 tokens, 4 experts each, in a buffer with room for 32 tokens
        {"name": "grouped_decode", "op": "grouped", "tokens": 24, "rows": 128, "used": 96, "experts": 32, "active": 29,
         "n": 4096, "k": 2048, "fmt": "fp8", "y": "bf16", "gather": True},
        # a prompt of 2048 tokens, 4 experts each, unevenly loaded
        {"name": "grouped_prompt", "op": "grouped", "tokens": 2048, "rows": 8192, "used": 8192, "experts": 32, "active": 32,
         "n": 4096, "k": 2048, "fmt": "fp8", "y": "bf16", "gather": True},
        # the down projections of 8 experts, one of them idle, 4-bit activations already in expert order
        {"name": "grouped_down", "op": "grouped", "tokens": 3001, "rows": 3001, "used": 3001, "experts": 8, "active": 7,
         "n": 2048, "k": 5632, "fmt": "fp4", "y": "f32", "gather": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quant", "norm", "linear", "linear", "grouped", "grouped"])
    fmt = rng.choice(["fp8", "fp4"])
    k = BLOCK * _log(rng, 8, 344)                      # 256 .. 11008
    if op == "quant":
        return {"op": op, "rows": min(_log(rng, 1, 16384), 45_000_000 // k), "k": k, "fmt": fmt,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "norm":
        return {"op": op, "rows": min(_log(rng, 1, 16384), 33_000_000 // k), "k": k, "fmt": fmt,
                "dtype": rng.choice(["bf16", "f16"]), "residual": rng.random() < 0.75}
    # 4-bit activations multiply exactly on any output; 8-bit ones are followed by a bf16 layer
    y = "bf16" if fmt == "fp8" else rng.choice(["bf16", "f32"])
    if op == "linear":
        m, n = _log(rng, 1, 4096), _log(rng, 64, 11008)
        return {"op": op, "m": m, "n": n, "k": k, "fmt": fmt, "y": y}
    experts = rng.choice([4, 8, 16, 32, 64])
    n = _log(rng, 128, 4096)
    k = min(k, BLOCK * 176)                            # to 5632
    tokens = _log(rng, 1, 2048)
    gather = rng.random() < 0.6
    used = tokens * rng.randint(1, min(4, experts)) if gather else tokens
    active = rng.randint(1, min(experts, used))
    rows = used + (rng.randint(1, 64) if rng.random() < 0.3 else 0)
    return {"op": op, "tokens": tokens if gather else rows, "rows": rows, "used": used, "experts": experts,
            "active": active, "n": n, "k": k, "fmt": fmt, "y": y, "gather": gather}


# ------------------------------------------------------------------ inputs
def _activations(gen, rows, k):
    """Hidden states: unit normal, tokens of different size, a few channels much larger than the rest."""
    x = torch.randn((rows, k), generator=gen, device="cuda")
    x *= 0.5 + torch.rand((rows, 1), generator=gen, device="cuda")
    x[:, torch.randint(0, k, (max(1, k // 256),), generator=gen, device="cuda")] *= 12.0
    return x


def _weights(gen, shape):
    """Linear weights: normal at sigma 0.02, rows of different size."""
    w = torch.randn(shape, generator=gen, device="cuda")
    w *= 0.01 + 0.02 * torch.rand(shape[:-1] + (1,), generator=gen, device="cuda")
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 40) + 17)
    op, fmt, k = case["op"], case["fmt"], case["k"]
    s = {"op": op, "fmt": fmt}
    if op in ("quant", "norm"):
        rows, dtype = case["rows"], DTYPE[case["dtype"]]
        x = _activations(gen, rows, k)
        if op == "quant":
            if rows >= 4:
                x[rows // 2, : k // 2] = 0.0            # whole blocks of zeros
            s["x"] = x.to(dtype)
            return s
        s["x"] = x.to(dtype)
        s["gamma"] = (1.0 + 0.1 * torch.randn((k,), generator=gen, device="cuda")).to(dtype)
        s["residual"] = (4.0 * _activations(gen, rows, k)).to(dtype) if case["residual"] else None
        return s
    s["y"] = DTYPE[case["y"]]
    if op == "linear":
        s["xq"], s["xs"] = _quantize(_activations(gen, case["m"], k), fmt)
        s["wq"], s["ws"] = _quantize(_weights(gen, (case["n"], k)), "fp4")
        return s
    tokens, rows, used = case["tokens"], case["rows"], case["used"]
    experts, active = case["experts"], case["active"]
    host = torch.Generator()
    host.manual_seed(int(seed) + 5)
    # the experts in use have a row at least; the others' load falls off as routers' loads do
    ids = torch.randperm(experts, generator=host)[:active]
    load = torch.exp(0.8 * torch.randn((active,), generator=host))
    counts = torch.zeros(experts, dtype=torch.int64)
    counts[ids] = 1
    if used > active:
        pick = torch.multinomial(load, used - active, replacement=True, generator=host)
        counts.index_add_(0, ids[pick], torch.ones_like(pick))
    offsets = torch.zeros(experts + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    s["offsets"], s["most"] = offsets.cuda(), int(counts.max())
    s["xq"], s["xs"] = _quantize(_activations(gen, tokens, k), fmt)
    s["rows"] = None
    if case["gather"]:
        s["rows"] = torch.randint(0, tokens, (rows,), generator=gen, device="cuda").to(torch.int32)
    s["wq"], s["ws"] = _quantize(_weights(gen, (experts, case["n"], k)), "fp4")
    return s


# ------------------------------------------------------------------ plain forms
def _scaled(v, e):
    """v * 2**e in fp32, e int32: two exact powers of two (a device pow() need not be exact)."""
    h = e >> 1
    return v * ((h + 127) << 23).view(torch.float32) * ((e - h + 127) << 23).view(torch.float32)


def _quantize(x, fmt):
    """Elements and scales of the MX form of x [..., k], in 32 bits."""
    emax, bits, emin, largest = GRID[fmt]
    v = x.float().reshape(x.shape[:-1] + (x.shape[-1] // BLOCK, BLOCK))
    a = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(a)[1].to(torch.int32) - 1 - emax + 127        # floor(log2 a) - emax, biased
    e = torch.where(a == 0, torch.zeros_like(e), e).clamp(0, 254)
    u = _scaled(v, 127 - e)
    m = u.abs()
    q = torch.frexp(m)[1].to(torch.int32) - 1
    q = torch.where(m == 0, torch.full_like(q, emin), q).clamp_min(emin) - bits   # exponent of the last place
    n = torch.round(_scaled(m, -q))                           # ties to even
    m = _scaled(n, q).clamp_max(largest)
    # the code of a value: the values of one sign are numbered in order
    f = torch.frexp(m)[1].to(torch.int32) - 1
    f = torch.where(m == 0, torch.full_like(f, emin), f).clamp_min(emin)
    low = _scaled(m, bits - f).to(torch.int32)                # with the leading 1 of a normal
    code = low + (f - emin) * (1 << bits)
    code = code + torch.signbit(u).to(torch.int32) * (8 if fmt == "fp4" else 128)
    code = code.reshape(x.shape)
    if fmt == "fp4":
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code.to(torch.uint8).contiguous(), e.squeeze(-1).to(torch.uint8).contiguous()


def _values(q, scales, fmt):
    """The fp32 values of an MX form."""
    if fmt == "fp4":
        c = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[:-1] + (2 * q.shape[-1],)).to(torch.int32)
    else:
        c = q.to(torch.int32)
    _, bits, emin, _ = GRID[fmt]
    sign = 8 if fmt == "fp4" else 128
    mag = c & (sign - 1)
    e, low = mag >> bits, mag & ((1 << bits) - 1)
    low = torch.where(e > 0, low + (1 << bits), low)
    v = _scaled(low.float(), e.clamp_min(1) - 1 + emin - bits)
    v = torch.where(c >= sign, -v, v)
    b = scales.to(torch.int32).unsqueeze(-1) - 127
    return _scaled(v.reshape(b.shape[:-1] + (BLOCK,)), b).reshape(v.shape)


def _plain(s):
    op, fmt = s["op"], s["fmt"]
    if op == "quant":
        return {"values": _values(*_quantize(s["x"], fmt), fmt).to(torch.bfloat16)}
    if op == "norm":
        x = s["x"]
        h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
        r = h.float()
        y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["gamma"].float()
        out = {"values": _values(*_quantize(y, fmt), fmt).to(torch.bfloat16)}
        if s["residual"] is not None:
            out["residual"] = h
        return out
    x, w = _values(s["xq"], s["xs"], fmt), _values(s["wq"], s["ws"], "fp4")
    if op == "linear":
        return {"y": torch.matmul(x, w.t()).to(s["y"])}
    # rows of an expert side by side, padded to the longest expert's
    experts, n, k = w.shape
    rows = x.shape[0] if s["rows"] is None else s["rows"].shape[0]
    t = torch.arange(rows, device=x.device)
    e = torch.searchsorted(s["offsets"][1:].long(), t, right=True)
    live = e < experts
    e = e.clamp_max(experts - 1)
    at = (t - s["offsets"].long()[e]).clamp(0, s["most"] - 1)
    src = t if s["rows"] is None else s["rows"].long()
    xp = torch.zeros((experts, s["most"], k), device=x.device)
    xp.index_put_((e, at), x[src] * live.unsqueeze(-1), accumulate=True)
    y = torch.bmm(xp, w.transpose(1, 2))[e, at] * live.unsqueeze(-1)
    return {"y": y.to(s["y"])}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import weight_only_bit_unpack_amd as w4
    op = s["op"]
    fmt = w4.W4_MXFP4 if s["fmt"] == "fp4" else w4.W4_MXFP8
    if op == "quant":
        q, scales = w4.w4_mx_quantize(s["x"], fmt)
        return {"values": w4.w4_mx_dequant(q, scales, fmt)}
    if op == "norm":
        q, scales, residual = w4.w4_mx_rmsnorm(s["x"], s["gamma"], EPS, fmt, residual=s["residual"])
        out = {"values": w4.w4_mx_dequant(q, scales, fmt)}
        if residual is not None:
            out["residual"] = residual
        return out
    if op == "linear":
        return {"y": w4.w4_mx_linear(s["xq"], s["xs"], s["wq"], s["ws"], fmt, y_dtype=s["y"])}
    return {"y": w4.w4_mx_grouped_linear(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], fmt,
                                         rows=s["rows"], y_dtype=s["y"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _levels(fmt):
    """Every non-negative element value in order, from the format's definition."""
    if fmt == "fp4":
        return [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    sub = [i / 8 * 2.0 ** -6 for i in range(8)]
    return sub + [(1 + i / 8) * 2.0 ** (e - 7) for e in range(1, 16) for i in range(8)][:-1]


def _pow2(e):
    """2**e in fp64 for whole numbers e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round(v, fmt):
    """fp64 [..., k] -> the fp64 values of its MX form: nearest level of each block's scaled grid."""
    lev = torch.tensor(_levels(fmt), dtype=torch.float64, device=v.device)
    mid = (lev[1:] + lev[:-1]) / 2
    b = v.reshape(-1, BLOCK)
    a = b.abs().amax(1, keepdim=True)
    e = torch.floor(torch.log2(a.clamp_min(1e-300)))
    e = torch.where(_pow2(e + 1) <= a, e + 1, torch.where(_pow2(e) > a, e - 1, e))
    scale = _pow2((e - GRID[fmt][0]).clamp(-127, 127))
    scale = torch.where(a == 0, torch.full_like(scale, 2.0 ** -127), scale)
    m = b.abs() / scale
    lo = torch.bucketize(m, mid)                    # midpoints strictly below m: a tie keeps the lower level
    tie = m == mid[lo.clamp_max(len(mid) - 1)]
    lo = torch.where(tie & (lo % 2 == 1), lo + 1, lo)
    return (torch.sign(b) * lev[lo] * scale).reshape(v.shape)


def _exact_values(q, scales, fmt):
    lev = _levels(fmt)
    table = torch.tensor(lev + ([float("nan")] if fmt == "fp8" else []), dtype=torch.float64, device=q.device)
    table = torch.cat((table, -table))
    if fmt == "fp4":
        v = torch.empty(q.shape[:-1] + (2 * q.shape[-1],), dtype=torch.float64, device=q.device)
        v[..., 0::2], v[..., 1::2] = table[(q % 16).long()], table[(q // 16).long()]
    else:
        v = table[q.long()]
    return v * _pow2(scales.int() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = s["op"], s["fmt"]
    if op == "quant":
        return {"values": _exact_round(s["x"].double(), fmt)}
    if op == "norm":
        out = {}
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["residual"] = h
            # the sum as it is stored: two values of 16 bits add exactly in 64, and round once
            h = h.to(s["x"].dtype).double()
        y = h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / h.shape[-1] + EPS) * s["gamma"].double()
        out["values"] = _exact_round(y, fmt)
        return out
    x = _exact_values(s["xq"], s["xs"], fmt)
    if op == "linear":
        return {"y": x @ _exact_values(s["wq"], s["ws"], "fp4").t()}
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    y = torch.zeros((x.shape[0], case["n"]), dtype=torch.float64, device=x.device)
    ends = s["offsets"].tolist()
    for e in range(case["experts"]):
        if ends[e + 1] > ends[e]:
            y[ends[e]:ends[e + 1]] = x[ends[e]:ends[e + 1]] @ _exact_values(s["wq"][e], s["ws"][e], "fp4").t()
    return {"y": y}


# ------------------------------------------------------------------ work
def work(case):
    op, k = case["op"], case["k"]
    per = (0.5 if case["fmt"] == "fp4" else 1.0) + 1 / BLOCK        # bytes of an element with its share of the scale
    w = 0.5 + 1 / BLOCK
    if op == "quant":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["rows"] * k * (size + per + 2), "flops": 4 * case["rows"] * k}
    if op == "norm":
        moved = 2 + per + 2 + (4 if case["residual"] else 0)
        return {"bytes": case["rows"] * k * moved + 2 * k, "flops": 6 * case["rows"] * k}
    size = 4 if case["y"] == "f32" else 2
    if op == "linear":
        m, n = case["m"], case["n"]
        return {"bytes": m * k * per + n * k * w + m * n * size, "flops": 2 * m * n * k}
    n, used = case["n"], case["used"]
    read = min(case["tokens"], used) * k * per + case["active"] * n * k * w
    return {"bytes": read + case["rows"] * n * size, "flops": 2 * used * n * k}
