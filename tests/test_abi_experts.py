"""Argument checks of the entry points of a layer of experts (no GPU: they come before any device work), and the tests'
64-bit gradient forms against differences."""

from __future__ import annotations

import pytest
import torch

import experts_ref as ref
import persistent_gemm_amd as pg

P = [0x10000000 * (i + 1) for i in range(12)]       # addresses far from each other
ARG, ALIGN = 1, 2


def _status(name, base, kw):
    a = dict(base)
    a.update(kw)
    return getattr(pg.load(), name)(*a.values(), None)


ROUTE = dict(logits=P[0], elem=1, normalize=1, experts=P[1], weights=P[2], offsets=P[3], slots=P[4], rows=P[5], work=P[6],
             T=100, E=16, k=2)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("logits", "experts", "weights", "offsets", "slots", "rows", "work")],
    (dict(elem=3), ARG), (dict(T=0), ARG), (dict(E=0), ARG), (dict(k=0), ARG), (dict(k=17), ARG), (dict(E=1025), ARG),
    (dict(E=64, k=33), ARG), (dict(T=1 << 30), ARG), (dict(T=1 << 31), ARG),
    (dict(logits=P[0] + 2), ALIGN), (dict(elem=0, logits=P[0] + 1), ALIGN), (dict(slots=P[4] + 2), ALIGN), (dict(work=P[6] + 1), ALIGN),
    (dict(rows=P[0] + 64), ARG), (dict(weights=P[1] + 60), ARG), (dict(work=P[3] + 64), ARG),
])
def test_route_checks(kw, status):
    assert _status("sk_moe_route", ROUTE, kw) == status


def test_route_work_bytes():
    f = pg.load().sk_moe_route_work_bytes
    assert f(1, 64) == 0 and f(64, 64) == 0 and f(65, 64) > 0 and f(0, 8) == 0 and f(100, 0) == 0 and f(100, 1025) == 0
    for T in (65, 1000, 32768, 32769, 1 << 20, 123456789):
        assert 0 < f(T, 16) <= 256 * 64          # at most 256 workgroups


ROUTE_GRAD = dict(dweights=P[0], logits=P[1], elem=0, normalize=0, experts=P[2], weights=P[3], dlogits=P[4], T=8, E=16, k=2)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("dweights", "logits", "experts", "weights", "dlogits")],
    (dict(elem=3), ARG), (dict(T=0), ARG), (dict(k=17), ARG), (dict(dlogits=P[4] + 1), ALIGN), (dict(dweights=P[0] + 2), ALIGN),
    (dict(dlogits=P[1]), ARG), (dict(dlogits=P[3] + 32), ARG),
])
def test_route_backward_checks(kw, status):
    assert _status("sk_moe_route_backward", ROUTE_GRAD, kw) == status


COMBINE = dict(y=P[0], elem=0, slots=P[1], weights=P[2], out=P[3], T=8, k=2, R=16, D=64)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("y", "slots", "out")],
    (dict(elem=-1), ARG), (dict(T=0), ARG), (dict(k=33), ARG), (dict(R=0), ARG), (dict(R=1 << 31), ARG), (dict(D=(1 << 22) + 1), ARG),
    (dict(y=P[0] + 1), ALIGN), (dict(elem=1, out=P[3] + 2), ALIGN), (dict(weights=P[2] + 2), ALIGN), (dict(out=P[0] + 128), ARG),
])
def test_combine_checks(kw, status):
    assert _status("sk_moe_combine", COMBINE, kw) == status


COMBINE_GRAD = dict(dout=P[0], y=P[1], elem=0, slots=P[2], weights=P[3], offsets=P[4], dy=P[5], dweights=P[6], T=8, k=2, R=16, D=64,
                    E=4)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("dout", "y", "slots", "dy")],
    (dict(E=0), ARG), (dict(E=1025), ARG), (dict(T=0), ARG), (dict(R=0), ARG), (dict(dy=P[5] + 2), ALIGN), (dict(dweights=P[6] + 2), ALIGN),
    (dict(dy=P[1]), ARG), (dict(dweights=P[3]), ARG), (dict(dy=P[0]), ARG),
])
def test_combine_backward_checks(kw, status):
    assert _status("sk_moe_combine_backward", COMBINE_GRAD, kw) == status


GROUPED = dict(A=P[0], B=P[1], elem=0, offsets=P[2], rows=P[3], bias=P[4], C=P[5], R=16, T=8, E=4, N=33, K=64, tail=0)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("A", "B", "offsets", "C")],
    (dict(elem=1), ARG), (dict(rows=None), ARG), (dict(R=0), ARG), (dict(T=0), ARG), (dict(E=0), ARG), (dict(E=1025), ARG), (dict(N=0), ARG),
    (dict(N=(1 << 22) + 1), ARG), (dict(K=(1 << 21) + 8), ARG), (dict(R=1 << 31), ARG),
    (dict(T=1 << 20, K=1024), ARG), (dict(T=(1 << 20) - 2, K=1024), ARG),           # rows of an A of 2 GiB, and of 4 KiB less
    (dict(K=68), ALIGN), (dict(A=P[0] + 8), ALIGN), (dict(B=P[1] + 2), ALIGN), (dict(C=P[5] + 1), ALIGN), (dict(rows=P[3] + 2), ALIGN),
    (dict(C=P[0] + 16), ARG), (dict(C=P[3]), ARG), (dict(bias=P[5] + 8), ARG),
])
def test_grouped_checks(kw, status):
    assert _status("sk_gemm_grouped", GROUPED, kw) == status


GROUPED_GRAD = dict(dC=P[0], A=P[1], B=P[2], elem=2, offsets=P[3], rows=P[4], dA=P[5], dB=P[6], dbias=P[7], R=16, T=8, E=4, N=64, K=64)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("dC", "A", "B", "offsets")], (dict(dA=None, dB=None, dbias=None), ARG),
    (dict(elem=1), ARG), (dict(rows=None), ARG), (dict(N=36), ALIGN), (dict(K=36), ALIGN), (dict(dC=P[0] + 8), ALIGN), (dict(dA=P[5] + 1), ALIGN),
    (dict(N=(1 << 21) + 8), ARG), (dict(dA=P[0]), ARG), (dict(dB=P[5] + 64), ARG), (dict(dbias=P[1]), ARG),
])
def test_grouped_backward_checks(kw, status):
    assert _status("sk_gemm_grouped_backward", GROUPED_GRAD, kw) == status


QUANT = dict(w=P[0], elem=1, q=P[1], scale=P[2], scale_elem=0, zero=P[3], E=1, N=8, K=128, group=64)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("w", "q", "scale")], (dict(elem=3), ARG), (dict(scale_elem=1), ARG), (dict(group=16), ARG), (dict(group=0), ARG),
    (dict(K=96), ARG), (dict(N=0), ARG), (dict(E=0), ARG), (dict(E=1025), ARG), (dict(w=P[0] + 2), ALIGN), (dict(q=P[1] + 8), ALIGN),
    (dict(scale=P[2] + 1), ALIGN), (dict(q=P[0] + 16), ARG), (dict(zero=P[2]), ARG),
])
def test_quantize_checks(kw, status):
    assert _status("sk_quantize_w4", QUANT, kw) == status


DEQUANT = dict(q=P[0], scale=P[1], scale_elem=0, zero=None, out=P[2], E=1, N=8, K=128, group=64)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("q", "scale", "out")], (dict(scale_elem=1), ARG), (dict(group=48), ARG), (dict(K=32), ARG),
    (dict(out=P[2] + 2), ALIGN), (dict(q=P[0] + 4), ALIGN), (dict(out=P[0]), ARG),
])
def test_dequantize_checks(kw, status):
    assert _status("sk_dequantize_w4", DEQUANT, kw) == status


W4 = dict(x=P[0], q=P[1], scale=P[2], zero=P[3], elem=0, offsets=P[4], rows=P[5], bias=P[6], C=P[7], M=16, T=8, E=4, N=33, K=128, group=64,
          tail=0)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, ARG) for n in ("x", "q", "scale", "C", "rows", "offsets")], (dict(elem=1), ARG), (dict(group=256), ARG), (dict(K=96), ARG),
    (dict(M=0), ARG), (dict(E=1025), ARG), (dict(offsets=None, rows=None, T=16), ARG),      # several experts without offsets
    (dict(offsets=None, rows=None, E=1), ARG), (dict(offsets=None, rows=None, E=1, M=(1 << 20) + 1, T=(1 << 20) + 1), ARG),
    (dict(x=P[0] + 8), ALIGN), (dict(q=P[1] + 8), ALIGN), (dict(C=P[7] + 1), ALIGN),
    (dict(C=P[0]), ARG), (dict(C=P[2] + 16), ARG), (dict(bias=P[7]), ARG),
])
def test_w4_checks(kw, status):
    assert _status("sk_gemm_w4", W4, kw) == status


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses():
    with pytest.raises(TypeError):
        pg.moe_route(None, 2)
    with pytest.raises(ValueError):
        pg.moe_route(torch.zeros(3), 2)
    for call in (lambda x: pg.moe_route(x, 2), lambda x: pg.quantize_w4(x, 32),
                 lambda x: pg.gemm_grouped(x, x[None], torch.zeros(2, dtype=torch.int32)),
                 lambda x: pg.moe_combine(x, torch.zeros(4, 2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="expected a GPU"):
            call(torch.zeros(4, 32))


# ---------------------------------------------------------------- the tests' own gradient forms

def _differences(f, x, h=1e-6):
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).reshape(-1)
        d[i] = h
        d = d.reshape(x.shape)
        out.reshape(-1)[i] = (f(x + d) - f(x - d)) / (2 * h)
    return out


@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_form(normalize):
    g = torch.Generator().manual_seed(1)
    x, d = torch.randn(4, 7, generator=g, dtype=torch.float64), torch.randn(4, 3, generator=g)
    ids = ref.route(x, 3, normalize)[0]
    f = lambda v: float((ref.route_weights(v, ids, normalize) * d.double()).sum())      # noqa: E731
    assert torch.allclose(ref.route_grad(d, x, ids, normalize), _differences(f, x), atol=1e-8)


def test_product_and_sum_gradient_forms():
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)       # noqa: E731
    A, B, bias, dC = r(4, 8), r(3, 5, 8), r(3, 5), r(7, 5)
    offsets, rows = torch.tensor([0, 3, 3, 6], dtype=torch.int32), torch.tensor([0, 1, 3, 1, 2, 3, -1], dtype=torch.int32)
    loss = lambda a, b, c: float((ref.grouped(a, b, offsets, c, rows)[0] * dC).sum())   # noqa: E731
    (dA, dB, db), _ = ref.grouped_grad(dC, A, B, offsets, rows)
    by_token = torch.zeros_like(A).index_add(0, rows.long()[:6], dA[:6])
    assert torch.allclose(by_token, _differences(lambda v: loss(v, B, bias), A), atol=1e-7)
    assert torch.allclose(dB, _differences(lambda v: loss(A, v, bias), B), atol=1e-7)
    assert torch.allclose(db, _differences(lambda v: loss(A, B, v), bias), atol=1e-7)
    y, w, d = r(6, 3), r(3, 2), r(3, 3)
    slots = torch.tensor([[4, 0], [-1, 2], [3, 6]], dtype=torch.int32)
    total = lambda v, u: float((ref.combine(v, slots, u)[0] * d).sum())     # noqa: E731
    dy, dw, _ = ref.combine_grad(d, y, slots, w)
    assert torch.allclose(dy, _differences(lambda v: total(v, w), y), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda v: total(y, v), w), atol=1e-8)
