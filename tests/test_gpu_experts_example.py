"""The example layer of experts: training and serving through the public calls, against the same layer in 64 bits."""

from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

# Elements are rounded to bf16, off by at most 2^-8 of themselves, at most eight times one after the other (u, twice in
# its square, y, out, dy, da, du, a row of dx), each time by all of a chain's earlier error and its own; the gradient of the logits
# is a difference whose parts are about as large as itself, which doubles what they bring.  The norm of the whole is then off
# by at most 16 of them.
BOUND = 16 * 2.0 ** -8


def _example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "experts.py")
    spec = importlib.util.spec_from_file_location("experts_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(v, x, ids):
    """The layer in 64 bits for given choices, one expert at a time, with autograd: v's tensors are its leaves."""
    logits = x @ v["router"].t()
    chosen = logits.gather(1, ids)
    w = torch.exp(chosen - chosen.amax(dim=1, keepdim=True))
    w = w / w.sum(dim=1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(len(v["W1"])):
        t, j = (ids == e).nonzero(as_tuple=True)
        r = torch.relu(x[t] @ v["W1"][e].t() + v["b1"][e])
        out = out.index_add(0, t, w[t, j, None] * ((r * r) @ v["W2"][e].t()))
    return out


def _layer(m, width, hidden, E, k, seed):
    layer = m.Experts(width, hidden, E, k, seed=seed)
    layer.p["b1"] += 0.1 * torch.randn(layer.p["b1"].shape, generator=torch.Generator().manual_seed(seed)).cuda()
    layer.cast()
    return layer


@pytest.mark.parametrize("tokens,width,hidden,E,k", [(130, 200, 648, 8, 2), (1, 64, 128, 8, 8), (300, 136, 264, 40, 6), (700, 128, 256, 2, 1)])
def test_gradients_follow_the_plain_layer(tokens, width, hidden, E, k):
    m = _example()
    layer = _layer(m, width, hidden, E, k, seed=3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(tokens, width, generator=g).to(torch.bfloat16)
    dout = torch.randn(tokens, width, generator=g).to(torch.bfloat16)
    out, saved = layer.forward(x.cuda())
    dx, grads = layer.backward(dout.cuda(), saved)
    leaves = {n: w.double().cpu().requires_grad_() for n, w in layer.v.items()}
    xl = x.double().requires_grad_()
    want = _plain(leaves, xl, saved[2].cpu().long()) + xl
    want.backward(dout.double())
    pairs = {"out": (out, want.detach()), "dx": (dx, xl.grad), **{n: (grads[n], leaves[n].grad) for n in leaves}}
    for name, (got, w) in pairs.items():
        got = got.double().cpu()
        assert got.shape == w.shape
        if k == 1 and name == "router":
            assert not got.any() and w.norm() < 1e-9          # (a single weight is always 1)
        else:
            assert (got - w).norm() <= BOUND * w.norm(), f"{name}: {((got - w).norm() / w.norm()).item()}"


def test_training_runs():
    m = _example()
    losses = m.train(m.Experts(128, 256, 8, 2, seed=1), 200, 3)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


@pytest.mark.parametrize("group,zero", [(32, False), (64, True), (128, True)])
def test_serving_follows_its_weights(group, zero):
    """Together and one token at a time, against 64 bits with the values that the 4-bit weights stand for."""
    m = _example()
    layer = _layer(m, 256, 384, 8, 2, seed=5)
    layer.quantize(group, zero)
    x = torch.randn(19, 256, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    together = layer.serve(x)
    apart = torch.cat([layer.serve(x[i:i + 1]) for i in range(len(x))])
    v = {n: w.double().cpu() for n, w in layer.v.items()}
    v["W1"], v["W2"] = (pg.dequantize_w4(*w).double().cpu() for w in (layer.w1, layer.w2))
    for got in (together, apart):
        ids = torch.cat([pg.moe_route(layer.logits(z), 2)[0] for z in ((x,) if got is together else x.split(1))])
        part = _plain(v, x.double().cpu(), ids.cpu().long())
        want = part + x.double().cpu()
        # (dequantised values are rounded once more, and the sum with x)
        assert (got.double().cpu() - want).norm() <= BOUND * part.norm() + 2.0 ** -8 * want.norm()
