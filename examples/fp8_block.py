#!/usr/bin/env python3
"""A residual block on block-scaled fp8 products, trained for a few steps and then run one token at a time.

    x -> rms_norm -> [W1, b1] -> relu^2 -> [W2] -> gated_norm (+ scaled residual x) -> out

Training takes both forms of each operand from one quantiser pass: the plain one for the product, the transposed
one for the gradient of the weights.  Weights are fp32, quantised in 128 x 128 tiles once a step (serving: once).  Serving
needs no gradients: the norm writes its fp8 output itself.

    python examples/fp8_block.py [--tokens T] [--width D] [--hidden H] [--steps N]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import persistent_gemm_amd as pg  # noqa: E402

EPS = 1e-6


class Fp8Block:
    def __init__(self, width, hidden, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.p = {
            "W1": torch.randn(hidden, width, generator=g, device=device) * width ** -0.5,
            "b1": torch.zeros(hidden, device=device),
            "W2": torch.randn(width, hidden, generator=g, device=device) * hidden ** -0.5,
            "norm": torch.ones(width, device=device),        # before the block
            "post": torch.ones(width, device=device),        # after it
            "gate": torch.full((width,), 0.25, device=device),
            "scale": torch.ones(width, device=device),       # of the residual
        }
        self.requantize()

    def requantize(self):
        """The weights' codes and the vectors in the activations' type; to be called when the weights have changed."""
        self.w1 = pg.quantize_fp8_block(self.p["W1"], "tile", transpose="both")
        self.w2 = pg.quantize_fp8_block(self.p["W2"], "tile", transpose="both")
        self.v = {k: self.p[k].to(torch.bfloat16) for k in ("b1", "norm", "post", "gate", "scale")}

    def forward(self, x):
        """out, and what the backward needs; x is bf16 [tokens, width]."""
        v = self.v
        y, rstd = pg.rms_norm(x, v["norm"], EPS)
        yq, ys, yt, yts = pg.quantize_fp8_block(y, transpose="both")
        u = pg.gemm_fp8_block(yq, self.w1[0], ys, self.w1[1], v["b1"])
        r = torch.relu(u)
        aq, as_, at, ats = pg.quantize_fp8_block(r * r, transpose="both")
        h = pg.gemm_fp8_block(aq, self.w2[0], as_, self.w2[1])
        out, rstd_h = pg.gated_norm(h, x, v["post"], v["gate"], v["scale"], EPS)
        return out, (x, rstd, yt, yts, r, at, ats, h, rstd_h)

    def backward(self, dout, saved):
        """(dx, gradients of the parameters)"""
        x, rstd, yt, yts, r, at, ats, h, rstd_h = saved
        v, g = self.v, {}
        dh, dx, g["post"], g["gate"], g["scale"], _ = pg.gated_norm_backward(dout, h, v["post"], rstd_h, v["gate"], x,
                                                                             v["scale"])
        da, g["W2"], _ = pg.gemm_fp8_block_backward(dh, at, ats, *self.w2[2:], need_dbias=False)
        du = 2 * da * r
        dy, g["W1"], g["b1"] = pg.gemm_fp8_block_backward(du, yt, yts, *self.w1[2:])
        dx, g["norm"] = pg.rms_norm_backward(dy, x, v["norm"], rstd, dresidual=dx)
        return dx, g

    def serve(self, x):
        """The block without what a backward needs: any number of tokens, one included."""
        v = self.v
        yq, ys, _ = pg.rms_norm(x, v["norm"], EPS, quantize=True)
        r = torch.relu(pg.gemm_fp8_block(yq, self.w1[0], ys, self.w1[1], v["b1"]))
        aq, as_ = pg.quantize_fp8_block(r * r)
        h = pg.gemm_fp8_block(aq, self.w2[0], as_, self.w2[1])
        return pg.gated_norm(h, x, v["post"], v["gate"], v["scale"], EPS)[0]


def train(block, tokens, steps, rate=0.1, seed=1, say=None):
    """Fits the block to another, randomly drawn, on fixed tokens; returns each step's loss."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width, hidden = block.p["W2"].shape
    x = torch.randn(tokens, width, generator=g, device="cuda").to(torch.bfloat16)
    target = Fp8Block(width, hidden, seed=seed + 1).serve(x).float()
    losses = []
    for step in range(steps):
        out, saved = block.forward(x)
        err = out.float() - target
        losses.append(err.square().mean().item())
        if say:
            say(f"step {step}: loss {losses[-1]:.5f}")
        _, grads = block.backward((2 / tokens * err).to(torch.bfloat16), saved)
        for k, p in block.p.items():
            p -= rate * grads[k].float()
        block.requantize()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    block = Fp8Block(a.width, a.hidden)
    train(block, a.tokens, a.steps, say=lambda s: print(s, flush=True))
    x = torch.randn(16, a.width, device="cuda").to(torch.bfloat16)
    together = block.serve(x)
    apart = torch.cat([block.serve(x[i:i + 1]) for i in range(len(x))])
    print(f"16 tokens together and one by one: largest difference {(together.float() - apart.float()).abs().max().item():.4g}")


if __name__ == "__main__":
    main()
