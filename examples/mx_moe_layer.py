#!/usr/bin/env python3
"""A mixture-of-experts feed-forward layer on the MX operators.

    python examples/mx_moe_layer.py [--tokens 64] [--hidden 2048] [--ffn 2816]
                                    [--experts 32] [--top 4]

The weights are quantized once to MXFP4 (4.25 bits each).  A call then runs

    residual add + RMS norm      -> MXFP8 activations, and the norm for the router
    router                       -> top experts of each token, rows in expert order
    grouped gate and up product  (one launch, rows gathered by index)
    silu(gate) * up              -> MXFP8 activations
    grouped down product
    weighted sum of each token's experts

with no host synchronisation, so that it can be captured in a HIP graph.  The
router's small product, the activation and the sum are torch operations.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_bit_unpack_amd as w4  # noqa: E402


class MxMoeLayer:
    """gamma [hidden]; router [experts, hidden]; gate_up [experts, 2 * ffn,
    hidden] (gate rows first); down [experts, hidden, ffn]: dense weights on
    the GPU, bf16.  hidden and ffn are multiples of 32."""

    def __init__(self, gamma, router, gate_up, down, top, eps=1e-5):
        self.gamma, self.router, self.top, self.eps = gamma, router, top, eps
        self.gate_up = self._quantize(gate_up)
        self.down = self._quantize(down)
        self.experts = router.shape[0]
        self.ids = torch.arange(self.experts + 1, device=gamma.device)

    @staticmethod
    def _quantize(w):
        q, s = w4.w4_mx_quantize(w.reshape(-1, w.shape[-1]), w4.W4_MXFP4)
        return q.view(w.shape[0], w.shape[1], -1), s.view(w.shape[0], w.shape[1], -1)

    def route(self, h):
        """Experts of each token: (weights [tokens, top], rows and offsets of the
        grouped products, place [tokens * top] of each choice among the rows)."""
        p, e = torch.topk(torch.softmax(h.float() @ self.router.float().t(), -1), self.top, -1)
        e, order = torch.sort(e.flatten(), stable=True)
        rows = (order // self.top).to(torch.int32)
        offsets = torch.searchsorted(e, self.ids).to(torch.int32)
        place = torch.empty_like(order)
        place[order] = torch.arange(order.numel(), device=order.device)
        return p / p.sum(-1, keepdim=True), rows, offsets, place

    def __call__(self, x, residual):
        """x, residual bf16 [tokens, hidden] -> (layer's output, the new residual)."""
        h = torch.empty_like(x)
        q, s, residual = w4.w4_mx_rmsnorm(x, self.gamma, self.eps, w4.W4_MXFP8, residual=residual, y=h)
        p, rows, offsets, place = self.route(h)
        a = w4.w4_mx_grouped_linear(q, s, *self.gate_up, offsets, rows=rows, y_dtype=torch.bfloat16)
        gate, up = a.float().chunk(2, -1)
        q, s = w4.w4_mx_quantize((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), w4.W4_MXFP8)
        y = w4.w4_mx_grouped_linear(q, s, *self.down, offsets, y_dtype=torch.bfloat16)
        # each token's experts in the router's order: the same sum every time
        y = (y[place].float().view(*p.shape, -1) * p.unsqueeze(-1)).sum(1)
        return y.to(torch.bfloat16), residual


def random_layer(hidden, ffn, experts, top, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, sigma=0.02: (torch.randn(s, generator=g, device="cuda") * sigma).to(torch.bfloat16)
    return dict(gamma=(1 + r(hidden, sigma=0.1).float()).to(torch.bfloat16), router=r(experts, hidden),
                gate_up=r(experts, 2 * ffn, hidden), down=r(experts, hidden, ffn), top=top)


def main():
    ap = argparse.ArgumentParser()
    for name, default in (("tokens", 64), ("hidden", 2048), ("ffn", 2816), ("experts", 32), ("top", 4)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    weights = random_layer(a.hidden, a.ffn, a.experts, a.top)
    layer = MxMoeLayer(**weights)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").to(torch.bfloat16)
    residual = 4 * torch.randn((a.tokens, a.hidden), generator=g, device="cuda").to(torch.bfloat16)
    y, _ = layer(x, residual)

    # the same layer with the bf16 weights and activations, in fp32
    h = (x.float() + residual.float()).to(torch.bfloat16).float()
    h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + layer.eps) * layer.gamma.float()
    p, rows, offsets, place = layer.route(h.to(torch.bfloat16))
    dense = torch.zeros((rows.numel(), a.hidden), device="cuda")
    ends = offsets.tolist()
    for e in range(a.experts):
        t = slice(ends[e], ends[e + 1])
        gate, up = (h[rows[t].long()] @ weights["gate_up"][e].float().t()).chunk(2, -1)
        dense[t] = (torch.nn.functional.silu(gate) * up) @ weights["down"][e].float().t()
    dense = (dense[place].view(*p.shape, -1) * p.unsqueeze(-1)).sum(1)
    err = ((y.float() - dense).norm() / dense.norm()).item()

    for _ in range(5):
        layer(x, residual)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(50):
        layer(x, residual)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t) / 50 * 1e6
    print(f"{a.tokens} tokens, hidden {a.hidden}, ffn {a.ffn}, top {a.top} of {a.experts} experts: {us:.0f} us a layer; "
          f"error against the unquantized layer {err:.3f} (4-bit weights, 8-bit activations)")


if __name__ == "__main__":
    main()
