"""The example block: training and serving through the public calls, against the same block in 64 bits."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch


pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "fp8_block.py")
    spec = importlib.util.spec_from_file_location("fp8_block_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(block, x):
    """The block in 64 bits, nothing quantised, with autograd."""
    p = {k: v.double().cpu().requires_grad_() for k, v in block.p.items()}
    x = x.double().cpu().requires_grad_()
    unit = lambda z: z * (z.square().mean(dim=1, keepdim=True) + 1e-6).rsqrt()
    r = torch.relu((unit(x) * p["norm"]) @ p["W1"].t() + p["b1"])
    out = p["scale"] * x + p["gate"] * (unit((r * r) @ p["W2"].t()) * p["post"])
    return out, x, p


def test_gradients_follow_the_plain_block():
    """An operand's code is off by at most 2^-4 of itself (half a step of E4M3), evenly up and down, so by 2^-4 / sqrt(3)
    at the root of the mean square; a chain of six quantised operands (y, W1, r^2, W2, dh, du) adds their squares: 0.09,
    twice that for the square of r, whose error counts double.  The direction of each gradient and of the output is within
    0.25 of the plain one's."""
    m = _example()
    block = m.Fp8Block(200, 650, seed=3)
    g = torch.Generator().manual_seed(4)
    for k in ("b1", "norm", "post", "gate", "scale"):
        block.p[k] += (0.1 * torch.randn(block.p[k].shape, generator=g)).cuda()
    block.requantize()
    x = torch.randn(130, 200, generator=g).to(torch.bfloat16)
    dout = torch.randn(130, 200, generator=g).to(torch.bfloat16)
    out, saved = block.forward(x.cuda())
    dx, grads = block.backward(dout.cuda(), saved)
    want, xr, p = _plain(block, x)
    want.backward(dout.double())
    pairs = {"out": (out, want.detach()), "dx": (dx, xr.grad), **{k: (grads[k], p[k].grad) for k in p}}
    for name, (got, w) in pairs.items():
        got = got.double().cpu()
        assert got.shape == w.shape
        assert (got - w).norm() <= 0.25 * w.norm(), f"{name}: {((got - w).norm() / w.norm()).item()}"


def test_training_lowers_the_loss():
    m = _example()
    losses = m.train(m.Fp8Block(256, 640, seed=1), 384, 8)
    assert losses[-1] < 0.9 * losses[0] and all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("width,hidden", [(256, 512), (333, 1000)])
def test_one_token_at_a_time(width, hidden):
    """One by one and together the norms and codes of y are the same bits; the products may add in another order, which
    moves u by one step of bf16 (2^-8 of it) and with that a code of r^2 by at most one step (2^-3 of it)."""
    m = _example()
    block = m.Fp8Block(width, hidden, seed=5)
    x = torch.randn(40, width, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    together = block.serve(x)
    apart = torch.cat([block.serve(x[i:i + 1]) for i in range(len(x))])
    a, b = together.double(), apart.double()
    assert ((a - b).norm(dim=1) <= 2.0 ** -3 * (b - x.double()).norm(dim=1) + 2.0 ** -8 * b.norm(dim=1)).all()
