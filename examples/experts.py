#!/usr/bin/env python3
"""A layer of experts, trained for a few steps in bf16 and then run one token at a time with 4-bit weights.

    x -> logits of the experts -> moe_route -> rows by expert
      -> [W1, b1] -> relu^2 -> [W2] -> moe_combine (by the choices' weights) + x -> out

The group sizes stay on the device, so that a step never waits for them.

    python examples/experts.py [--tokens T] [--width D] [--hidden H] [--experts E] [--choices K] [--steps N]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import persistent_gemm_amd as pg  # noqa: E402

BF = torch.bfloat16


class Experts:
    def __init__(self, width, hidden, experts, choices, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.k = choices
        self.p = {
            "router": torch.randn(experts, width, generator=g, device=device) * width ** -0.5,
            "W1": torch.randn(experts, hidden, width, generator=g, device=device) * width ** -0.5,
            "b1": torch.zeros(experts, hidden, device=device),
            "W2": torch.randn(experts, width, hidden, generator=g, device=device) * hidden ** -0.5,
        }
        self.cast()

    def cast(self):
        """The weights in the activations' type (the router's stay fp32); to be called when they have changed."""
        self.v = {n: w if n == "router" else w.to(BF) for n, w in self.p.items()}

    def quantize(self, group=128, zero=True):
        """4-bit forms of the experts' weights, for serve()."""
        self.w1 = pg.quantize_w4(self.v["W1"], group, zero=zero)
        self.w2 = pg.quantize_w4(self.v["W2"], group, zero=zero)

    def logits(self, x):
        return x.float() @ self.v["router"].t()

    def forward(self, x):
        """out, and what the backward needs; x is bf16 [tokens, width]."""
        v = self.v
        logits = self.logits(x)
        experts, weights, offsets, slots, rows = pg.moe_route(logits, self.k)
        r = torch.relu(pg.gemm_grouped(x, v["W1"], offsets, v["b1"], rows=rows))
        a = r * r
        y = pg.gemm_grouped(a, v["W2"], offsets)
        out = pg.moe_combine(y, slots, weights) + x
        return out, (x, logits, experts, weights, offsets, slots, rows, r, a, y)

    def backward(self, dout, saved):
        """(dx, gradients of the parameters)"""
        x, logits, experts, weights, offsets, slots, rows, r, a, y = saved
        v, g = self.v, {}
        dy, dweights = pg.moe_combine_backward(dout, y, slots, weights, offsets=offsets)
        da, g["W2"], _ = pg.gemm_grouped_backward(dy, a, v["W2"], offsets, need_dbias=False)
        dxr, g["W1"], g["b1"] = pg.gemm_grouped_backward(2 * da * r, x, v["W1"], offsets, rows=rows)
        dlogits = pg.moe_route_backward(dweights, logits, experts, weights)
        dx = dout + pg.moe_combine(dxr, slots)
        g["router"] = dlogits.t() @ x.float()
        return dx + (dlogits @ v["router"]).to(BF), g

    def serve(self, x):
        """The layer with quantize()'s weights: any few tokens, one included."""
        v = self.v
        _, weights, offsets, slots, rows = pg.moe_route(self.logits(x), self.k)
        r = torch.relu(pg.gemm_w4(x, *self.w1, v["b1"], offsets=offsets, rows=rows))
        return pg.moe_combine(pg.gemm_w4(r * r, *self.w2, offsets=offsets), slots, weights) + x


def train(layer, tokens, steps, lr=0.3, seed=1):
    """Losses of `steps` steps of gradient descent towards another layer's outputs."""
    device, width = layer.p["router"].device, layer.p["router"].shape[1]
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(tokens, width, generator=g, device=device).to(BF)
    want = x + torch.tanh(torch.randn(width, generator=g, device=device)) * x
    losses = []
    for _ in range(steps):
        out, saved = layer.forward(x)
        d = out.float() - want.float()
        losses.append(float((d * d).mean()))
        _, grads = layer.backward((2 / width * d).to(BF), saved)
        for n, w in layer.p.items():
            w -= lr * grads[n].float() / tokens
        layer.cast()
    return losses


def main():
    ap = argparse.ArgumentParser()
    for n, d in (("tokens", 1024), ("width", 1024), ("hidden", 2048), ("experts", 16), ("choices", 2), ("steps", 10)):
        ap.add_argument("--" + n, type=int, default=d)
    a = ap.parse_args()
    layer = Experts(a.width, a.hidden, a.experts, a.choices)
    losses = train(layer, a.tokens, a.steps)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    layer.quantize()
    x = torch.randn(4, a.width, device="cuda").to(BF)
    apart = torch.cat([layer.serve(x[i:i + 1]) for i in range(len(x))])
    whole = layer.forward(x)[0]
    err = ((apart.float() - whole.float()).norm() / (whole.float() - x.float()).norm()).item()
    print(f"4 tokens one by one with 4-bit weights: {err:.3f} of the layer's part away from bf16")


if __name__ == "__main__":
    main()
