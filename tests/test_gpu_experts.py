"""Routing, the weighted sum of experts' rows and products grouped by expert against 64-bit forms."""

from __future__ import annotations

import math

import pytest
import torch

import experts_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(seed, *shape, dtype=FP, scale=1.0):
    return (torch.randn(*shape, generator=_gen(seed)) * scale).to(dtype)


# ---------------------------------------------------------------- routing

def _check_route(x, k, normalize):
    got = pg.moe_route(x.cuda(), k, normalize=normalize)
    want = ref.route(x, k, normalize)
    for n, a, b in zip(("experts", "offsets", "slots", "rows"), (got[0], *got[2:]), (want[0], *want[2:])):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), n
    # the exponent's argument is off by half an fp32 step of itself, the exponential by 2 steps, and E terms are added
    far = torch.where(torch.isfinite(x.float()), x.float(), 0.0).abs().amax().item() * 2
    ref.assert_near(got[1], want[1], want[1].abs().nan_to_num() * (x.shape[1] + 8 + far) * ref.STEP32 + 2.0 ** -140, "weights")
    return got


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, FP), (1, 64, 6, FP), (3, 5, 5, HF), (7, 16, 16, FP), (64, 8, 2, BF), (255, 60, 6, FP), (256, 17, 4, HF),
    (257, 64, 8, FP), (300, 33, 2, BF), (513, 128, 8, FP), (700, 256, 8, FP), (65, 257, 3, HF), (40, 512, 32, FP),
    (33, 1024, 9, BF), (2000, 4, 1, FP), (64, 40, 8, HF), (65, 40, 8, BF), (127, 36, 4, FP),
])
def test_route(T, E, k, dtype, normalize):
    _check_route(_rand(T * 1000 + E, T, E, dtype=dtype, scale=2.0), k, normalize)


def test_route_many_tokens():
    # more tokens than 256 workgroups of 64 take
    T, E, k = 2 * 256 * 64 + 300, 8, 2
    x = _rand(5, T, E)
    got = pg.moe_route(x.cuda(), k)
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    assert torch.equal(got[0].cpu(), ids[:, :k].to(torch.int32))
    order = torch.sort(ids[:, :k].reshape(-1), stable=True).indices
    assert torch.equal(got[4].cpu().long(), order // k)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k)
    assert torch.equal(got[3].cpu().long().reshape(-1), place)
    assert torch.equal(got[2].cpu().long()[1:], torch.bincount(ids[:, :k].reshape(-1), minlength=E).cumsum(0))


@pytest.mark.parametrize("normalize", [True, False])
def test_route_ties_go_to_the_lowest_expert(normalize):
    g = _gen(11)
    x = torch.randint(-2, 3, (300, 70), generator=g).float()
    x[x == 0] = torch.where(torch.rand((x == 0).sum(), generator=g) < 0.5, 0.0, -0.0)     # both zeros are equal
    _check_route(x, 7, normalize)
    _check_route(torch.zeros(9, 1000), 32, normalize)


@pytest.mark.parametrize("normalize", [True, False])
def test_route_masks(normalize):
    x = _rand(12, 64, 20)
    x[0] = -math.inf                       # nothing left
    x[1, 3:] = -math.inf                   # fewer than k left
    x[2] = torch.finfo(FP).min             # the lowest value is a value
    x[3, :10], x[3, 10:] = torch.finfo(FP).min, -math.inf
    x[4, 5] = math.nan
    x[5, 7] = math.inf
    x[6, 2], x[6, 3] = -math.inf, math.nan
    x[7] = math.nan
    x[60:] = -math.inf                     # padding
    _check_route(x, 6, normalize)
    _check_route(torch.full((5, 3), -math.inf), 2, normalize)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, FP), (5, 8, 2, HF), (130, 60, 6, FP), (33, 256, 8, BF), (9, 700, 32, FP)])
def test_route_gradient(T, E, k, dtype, normalize):
    x = _rand(T + E, T, E, dtype=dtype)
    if T > 4:
        x[1] = -math.inf
        x[2, 1:] = -math.inf
    d = _rand(3, T, k)
    ids, w, *_ = pg.moe_route(x.cuda(), k, normalize=normalize)
    got = pg.moe_route_backward(d.cuda(), x.cuda(), ids, w, normalize=normalize)
    want = ref.route_grad(d, x, ids, normalize)
    assert got.dtype == dtype
    # the weights' error (test_route) times the gradients it meets, k of them added, and the last rounding
    size = d.abs().sum(dim=1, keepdim=True).double()
    ref.assert_near(got, want, ref.rounding(want, dtype) + size * (E + 2 * k + 20) * ref.STEP32)


# ---------------------------------------------------------------- the weighted sum

def _slots(seed, T, k, R, missing=0.2):
    g = _gen(seed)
    s = torch.randperm(R, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    return torch.where(torch.rand(T, k, generator=g) < missing, torch.tensor(-1, dtype=torch.int32), s)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,D,dtype", [(1, 1, 1, FP), (1, 2, 7, BF), (5, 3, 8, HF), (17, 2, 65, BF), (9, 32, 513, HF),
                                         (130, 4, 2051, BF), (33, 8, 1000, FP), (64, 2, 4096, BF)])
def test_combine(T, k, D, dtype, weighted):
    R = T * k + 3
    y, slots = _rand(T + D, R, D, dtype=dtype), _slots(D, T, k, R)
    w = _rand(2, T, k) if weighted else None
    got = pg.moe_combine(y.cuda(), slots.cuda(), None if w is None else w.cuda())
    want, mag = ref.combine(y, slots, w)
    ref.assert_near(got, want, ref.rounding(want, dtype) * 1.01 + mag * k * ref.STEP32)


def test_combine_slots_out_of_range_and_twice():
    y = _rand(1, 6, 40, dtype=BF)
    slots = torch.tensor([[0, 0], [6, -7], [2 ** 31 - 1, 5], [-2 ** 31, 3]], dtype=torch.int32)
    got = pg.moe_combine(y.cuda(), slots.cuda())
    want, mag = ref.combine(y, slots, None)
    ref.assert_near(got, want, ref.rounding(want, BF) * 1.01)


@pytest.mark.parametrize("form", ["weighted", "plain", "cleared"])
@pytest.mark.parametrize("T,k,D,dtype", [(1, 1, 1, FP), (3, 2, 7, BF), (5, 3, 8, HF), (17, 2, 65, BF), (9, 32, 513, HF),
                                         (130, 4, 2051, BF), (33, 8, 1000, FP), (64, 2, 4096, BF)])
def test_combine_gradient(T, k, D, dtype, form):
    x = _rand(D, T, 40)
    x[::3, 4:] = -math.inf                    # missing choices, and tokens without any
    x[1::4] = -math.inf
    ids, w, offsets, slots, rows = pg.moe_route(x.cuda(), k)
    R = T * k
    if form == "cleared":                      # rows that no slot names lie anywhere
        R += 5
        slots = torch.where(slots >= 0, slots + 2, slots)
    y, d = _rand(T + D, R, D, dtype=dtype), _rand(7, T, D, dtype=dtype)
    weights = None if form == "plain" else w
    dy, dw = pg.moe_combine_backward(d.cuda(), y.cuda(), slots, weights, offsets=None if form == "cleared" else offsets)
    want, want_w, mag = ref.combine_grad(d, y, slots.cpu(), None if weights is None else weights.cpu())
    ref.assert_near(dy, want, ref.rounding(want, dtype) + 2.0 ** -24 * want.abs() * 2, "dy")
    if form == "plain":
        assert dw is None
    else:
        ref.assert_near(dw, want_w, mag * (D + 1) * ref.STEP32 + 2.0 ** -140, "dweights")


# ---------------------------------------------------------------- products grouped by expert

def _offsets(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32)


def _check_grouped(counts, N, K, dtype, *, bias=False, gather=0, tail=0, seed=0):
    E, R = len(counts), sum(counts) + tail
    offsets = _offsets(counts)
    rows = torch.randint(0, gather, (R,), generator=_gen(seed)).to(torch.int32) if gather else None
    if tail and gather:
        rows[R - tail:] = -1
    A = _rand(seed + 1, gather or R, K, dtype=dtype)
    B = _rand(seed + 2, E, N, K, dtype=dtype, scale=K ** -0.5)
    b = _rand(seed + 3, E, N, dtype=dtype) if bias else None
    put = lambda t: None if t is None else t.cuda()      # noqa: E731
    got = pg.gemm_grouped(put(A), put(B), put(offsets), put(b), rows=put(rows))
    want, mag = ref.grouped(A, B, offsets, b, rows)
    # K products and the bias added in fp32 in any order, each addition off by at most a step, and one rounding
    bound = mag * (K + 1) * ref.STEP32
    ref.assert_near(got, want, ref.rounding(want, dtype) * 1.001 + bound)
    if tail:
        assert not got[R - tail:].any()
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    assert pg.gemm_grouped(put(A), put(B), put(offsets), put(b), rows=put(rows), out=out) is out
    assert torch.equal(out[:R - tail], got[:R - tail]) and bool((out[R - tail:] == 7.0).all())
    return got


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 1, 8), ([1], 16, 64), ([0, 1, 0], 5, 24), ([3, 0, 2, 1], 130, 72), ([16, 15, 17, 0, 1], 64, 128),
    ([40, 0, 3], 257, 136), ([255, 256, 257], 70, 200), ([700, 1], 300, 88), ([0, 0, 513], 515, 320),
])
def test_grouped(counts, N, K, dtype):
    _check_grouped(counts, N, K, dtype)
    _check_grouped(counts, N, K, dtype, bias=True, gather=max(1, sum(counts) // 2), tail=3, seed=9)


@pytest.mark.parametrize("N,K", [(8, 8), (100, 1000), (1000, 136)])
def test_grouped_many_experts(N, K):
    counts = torch.randint(0, 5, (300,), generator=_gen(3)).tolist()
    counts[70], counts[299] = 300, 0
    _check_grouped(counts, N, K, BF, bias=True, gather=50, tail=30)
    _check_grouped([0] * 200 + [5] + [0] * 823, N, K, HF)


def test_grouped_without_any_rows():
    got = _check_grouped([0, 0], 33, 64, BF, bias=True, tail=70)
    assert not got.any()


def test_grouped_large_tiles():
    _check_grouped([600, 0, 1100, 348], 520, 1096, BF, bias=True, gather=700, tail=5)
    _check_grouped([513, 2050], 777, 64, HF)


def test_grouped_rows_are_held_to_their_range():
    """Offsets and rows that are wrong give wrong rows, within the tensors."""
    A, B = _rand(1, 40, 64, dtype=BF).cuda(), _rand(2, 3, 72, 64, dtype=BF).cuda()
    rows = torch.tensor([-5, 1000, 2 ** 31 - 1, -2 ** 31] * 10, dtype=torch.int32).cuda()
    good = torch.tensor([0, 10, 20, 40], dtype=torch.int32).cuda()
    want, mag = ref.grouped(A, B, good, None, rows)
    got = pg.gemm_grouped(A, B, good, rows=rows)
    ref.assert_near(got, want, ref.rounding(want, BF) * 1.001 + mag * 65 * ref.STEP32)
    d = _rand(3, 40, 72, dtype=BF).cuda()
    for bad in ([0, 60, 20, 90], [-7, -3, 2 ** 31 - 1, -2 ** 31], [30, 20, 10, 0]):
        o = torch.tensor(bad, dtype=torch.int32).cuda()
        assert pg.gemm_grouped(A, B, o, rows=rows).shape == (40, 72)
        assert pg.gemm_grouped_backward(d, A, B, o, rows=rows)[1].shape == (3, 72, 64)


def _check_grouped_backward(counts, N, K, dtype, *, gather=0, tail=0, seed=0):
    E, R = len(counts), sum(counts) + tail
    offsets = _offsets(counts)
    rows = torch.randint(0, gather, (R,), generator=_gen(seed)).to(torch.int32) if gather else None
    if tail and gather:
        rows[R - tail:] = -1
    A, B = _rand(seed + 1, gather or R, K, dtype=dtype), _rand(seed + 2, E, N, K, dtype=dtype, scale=N ** -0.5)
    d = _rand(seed + 4, R, N, dtype=dtype)
    args = [None if t is None else t.cuda() for t in (d, A, B, offsets)]
    r = None if rows is None else rows.cuda()
    got = pg.gemm_grouped_backward(*args, rows=r)
    want, mag = ref.grouped_grad(d, A, B, offsets, rows)
    for n, g, w, m, terms in zip(("dA", "dB", "dbias"), got, want, mag, (N, max(counts), max(counts))):
        ref.assert_near(g, w, ref.rounding(w, dtype) * 1.001 + m * (terms + 1) * ref.STEP32, n)
    if tail:
        assert not got[0][R - tail:].any()
    for need in ("need_dA", "need_dB", "need_dbias"):       # each by itself: the same bits
        one = pg.gemm_grouped_backward(*args, rows=r, **({n: n == need for n in ("need_dA", "need_dB", "need_dbias")}))
        at = ("need_dA", "need_dB", "need_dbias").index(need)
        assert [x is None for x in one] == [i != at for i in range(3)]
        assert torch.equal(one[at], got[at])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8), ([0, 1, 0], 24, 16), ([3, 0, 2, 1], 136, 72), ([63, 64, 65, 0, 1], 64, 128), ([40, 0, 3], 264, 136),
    ([255, 256, 257], 72, 200), ([700, 1], 304, 520),
])
def test_grouped_backward(counts, N, K, dtype):
    _check_grouped_backward(counts, N, K, dtype)
    _check_grouped_backward(counts, N, K, dtype, gather=max(1, sum(counts) // 2), tail=3, seed=9)


def test_grouped_backward_many_experts():
    counts = torch.randint(0, 5, (150,), generator=_gen(3)).tolist()
    counts[70], counts[149] = 300, 0
    _check_grouped_backward(counts, 40, 72, BF, gather=50, tail=30)


def test_grouped_backward_large_tiles():
    _check_grouped_backward([600, 0, 1100, 348], 520, 1096, BF, gather=700, tail=5)
    _check_grouped_backward([513, 1050], 776, 264, HF)


def test_grouped_repeats():
    A, B = _rand(1, 1000, 520, dtype=BF).cuda(), _rand(2, 4, 400, 520, dtype=BF).cuda()
    offsets = _offsets([100, 500, 0, 400]).cuda()
    d = _rand(3, 1000, 400, dtype=BF).cuda()
    first = (pg.gemm_grouped(A, B, offsets), *pg.gemm_grouped_backward(d, A, B, offsets))
    for _ in range(3):
        again = (pg.gemm_grouped(A, B, offsets), *pg.gemm_grouped_backward(d, A, B, offsets))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
