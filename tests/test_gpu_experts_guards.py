"""Offsets, rows, slots and experts that are wrong: the calls of a layer of experts write within their outputs, and nothing else."""

from __future__ import annotations

import pytest
import torch

import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
LOW, HIGH = -2 ** 31, 2 ** 31 - 1
OFFSETS = [[0, 60, 20, 90], [-7, -3, HIGH, LOW], [30, 20, 10, 0], [HIGH, LOW, HIGH, LOW], [40, 40, 40, 40], [0, 0, 0, HIGH]]


class Guarded:
    """An output between guards of 64 KiB."""

    def __init__(self, *shape, dtype):
        n = torch.empty(shape, dtype=dtype, device="meta").numel() * dtype.itemsize
        self.all = torch.full((n + (1 << 17),), 0xA5, dtype=torch.uint8, device="cuda")
        self.at, self.end = 1 << 16, (1 << 16) + n
        self.t = self.all[self.at:self.end].view(dtype).view(shape)

    def ptr(self):
        return self.t.data_ptr()

    def whole(self):
        return bool((self.all[:self.at] == 0xA5).all()) and bool((self.all[self.end:] == 0xA5).all())


def _int(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rand(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _call(name, *args):
    p = [a.data_ptr() if isinstance(a, torch.Tensor) else a.ptr() if isinstance(a, Guarded) else a for a in args]
    assert getattr(pg.load(), name)(*p, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("R,N,K", [(40, 72, 64), (700, 520, 136)])
@pytest.mark.parametrize("offsets", OFFSETS)
def test_products_by_expert(offsets, R, N, K):
    T, E = 25, 3
    A, B, bias, d = _rand(1, T, K), _rand(2, E, N, K), _rand(3, E, N), _rand(4, R, N)
    o, rows = _int(*offsets), _int(*([-5, 1000, HIGH, LOW, 3] * R)[:R])
    for tail in (0, 1):
        C = Guarded(R, N, dtype=BF)
        _call("sk_gemm_grouped", A, B, 0, o, rows, bias, C, R, T, E, N, K, tail)
        assert C.whole()
    own = _rand(5, R, K)
    for a, r, t in ((A, rows, T), (own, None, R)):
        dA, dB, db = Guarded(R, K, dtype=BF), Guarded(E, N, K, dtype=BF), Guarded(E, N, dtype=BF)
        _call("sk_gemm_grouped_backward", d, a, B, 0, o, r, dA, dB, db, R, t, E, N, K)
        assert dA.whole() and dB.whole() and db.whole()
        alone = Guarded(E, N, dtype=BF)
        _call("sk_gemm_grouped_backward", d, a, B, 0, o, r, None, None, alone, R, t, E, N, K)
        assert alone.whole() and torch.equal(alone.t, db.t)


@pytest.mark.parametrize("R,N,K,group", [(40, 72, 128, 64), (300, 33, 96, 32)])
@pytest.mark.parametrize("offsets", OFFSETS)
def test_products_with_4_bit_weights(offsets, R, N, K, group):
    T, E = 25, 3
    q, s, z = pg.quantize_w4(_rand(2, E, N, K), group, zero=True)
    x, o, rows = _rand(1, T, K), _int(*offsets), _int(*([-5, 1000, HIGH, LOW, 3] * R)[:R])
    for tail in (0, 1):
        C = Guarded(R, N, dtype=BF)
        _call("sk_gemm_w4", x, q, s, z, 0, o, rows, None, C, R, T, E, N, K, group, tail)
        assert C.whole()


@pytest.mark.parametrize("D", [5, 72, 520])
def test_the_sum_of_rows_and_its_gradients(D):
    T, k, R, E = 9, 3, 20, 2
    y, d, w = _rand(1, R, D), _rand(2, T, D), _rand(3, T, k, dtype=FP)
    slots = _int(*([-1, R, HIGH, LOW, 0, R - 1, R + 7, 5, 2] * 3)).view(T, k)
    out = Guarded(T, D, dtype=BF)
    _call("sk_moe_combine", y, 0, slots, w, out, T, k, R, D)
    assert out.whole()
    for offsets in ([0, 3, HIGH], [0, 0, LOW], [0, 0, 7], None):
        dy, dw = Guarded(R, D, dtype=BF), Guarded(T, k, dtype=FP)
        _call("sk_moe_combine_backward", d, y, 0, slots, w, None if offsets is None else _int(*offsets), dy, dw, T, k, R, D, E)
        assert dy.whole() and dw.whole()


@pytest.mark.parametrize("E", [7, 64, 300])
def test_the_gradient_of_the_choice(E):
    T, k = 33, 3
    logits, w, dw = _rand(1, T, E, dtype=FP), _rand(2, T, k, dtype=FP), _rand(3, T, k, dtype=FP)
    ids = _int(*([-1, E, HIGH, LOW, 0, E - 1, E + 63, 1, 2] * 11)).view(T, k)
    for normalize in (0, 1):
        out = Guarded(T, E, dtype=FP)
        _call("sk_moe_route_backward", dw, logits, 1, normalize, ids, w, out, T, E, k)
        assert out.whole()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (64, 40, 8), (257, 33, 5), (40, 1024, 32)])
def test_the_choice(T, E, k):
    x = _rand(1, T, E, dtype=FP)
    i32 = torch.int32
    outs = [Guarded(T, k, dtype=i32), Guarded(T, k, dtype=FP), Guarded(E + 1, dtype=i32), Guarded(T, k, dtype=i32), Guarded(T * k, dtype=i32)]
    n = pg.load().sk_moe_route_work_bytes(T, E)
    work = Guarded(n // 4, dtype=i32) if n else None
    _call("sk_moe_route", x, 1, 1, *outs, work, T, E, k)
    assert all(o.whole() for o in outs) and (work is None or work.whole())
    assert torch.equal(outs[0].t.long(), torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k])
