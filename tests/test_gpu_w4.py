"""4-bit weights: codes, scales and zero points bit for bit, and products of few rows, against 64-bit forms."""

from __future__ import annotations

import math

import pytest
import torch

import experts_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _rand(seed, *shape, dtype=FP, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _check_codes(w, group, zero, dtype):
    q, s, z = pg.quantize_w4(w.cuda(), group, zero=zero, dtype=dtype)
    codes, scale, zeros = ref.quantize(w, group, zero, s.dtype)
    assert torch.equal(s.cpu().view(torch.int16)[~torch.isnan(scale)], scale.view(torch.int16)[~torch.isnan(scale)])
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(scale))
    assert torch.equal(ref.unpack(q), codes)
    assert (z is None) == (not zero)
    if zero:
        assert torch.equal(z.cpu(), zeros)
    got = pg.dequantize_w4(q, s, z)
    assert got.dtype == s.dtype
    # a scale of at most 11 bits times a whole number of 4 is exact in fp32, so one rounding gives the bits (an infinity
    # where the product is half a step past the type's largest number: the scale of a group of such numbers was rounded up)
    want = (ref.by_element(scale, group) * (codes.double() - ref.by_element(zeros, group))).float().to(s.dtype)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.equal(got.cpu().nan_to_num(5.0, math.inf, -math.inf), want.nan_to_num(5.0, math.inf, -math.inf))
    return q, s, z


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K,dtype,scale", [(1, 1, BF, None), (7, 3, HF, None), (65, 5, FP, None), (130, 2, FP, HF),
                                             (33, 9, BF, HF), (16, 1, HF, BF)])
def test_codes(N, K, dtype, scale, group, zero):
    _check_codes(_rand(N + K, N, K * group, dtype=dtype, scale=0.02), group, zero, scale)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_codes_at_borders(dtype, zero):
    """Values on and next to the borders between codes, all-zero, tiny, large and non-finite groups."""
    g = torch.Generator().manual_seed(4)
    w = torch.randint(-28, 29, (64, 128), generator=g).float() / 2      # quotients with the scale are halves at many
    w[:, 0], w[:, 1] = 14.0, -14.0
    if dtype == FP:
        w *= 1 + (torch.randint(-1, 2, w.shape, generator=g).float() * 2.0 ** -23)
    w = w.to(dtype)
    w[1], w[2] = 0, 0
    w[3] = torch.finfo(dtype).tiny / 2
    w[4, 7], w[5, 8], w[6, 9] = math.inf, -math.inf, math.nan
    w[7], w[8] = torch.finfo(dtype).max, torch.finfo(dtype).min
    w[9] = w[9].abs()                        # no negative value
    w[10] = -w[10].abs()
    for scale in (BF, HF):
        _check_codes(w, 64, zero, scale)


def test_codes_of_experts():
    w = _rand(3, 3, 40, 192, dtype=BF)
    q, s, z = pg.quantize_w4(w.cuda(), 64, zero=True)
    v = pg.dequantize_w4(q, s, z)
    for e in range(3):
        qe, se, ze = pg.quantize_w4(w[e].cuda(), 64, zero=True)
        assert torch.equal(q[e], qe) and torch.equal(s[e], se) and torch.equal(z[e], ze)
        assert torch.equal(v[e], pg.dequantize_w4(qe, se, ze))


def _check(M, N, K, group, zero, dtype, bias, seed=0):
    w = _rand(seed + M, N, K, dtype=dtype, scale=K ** -0.5)
    q, s, z = pg.quantize_w4(w.cuda(), group, zero=zero)
    x = _rand(seed + 1, M, K, dtype=dtype)
    b = _rand(seed + 2, N, dtype=dtype) if bias else None
    got = pg.gemm_w4(x.cuda(), q, s, z, None if b is None else b.cuda())
    want, mag = ref.w4(x, q, s, z, b, group)
    # 2 K terms, K / group products with a scale and the bias in fp32, each addition off by at most a step; one rounding
    ref.assert_near(got, want, ref.rounding(want, dtype) * 1.001 + mag * (2 * group + K // group + 8) * ref.STEP32)
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    assert pg.gemm_w4(x.cuda(), q, s, z, None if b is None else b.cuda(), out=out) is out
    assert torch.equal(out, got)


@pytest.mark.parametrize("dtype,zero,bias", [(BF, False, False), (BF, True, True), (HF, False, True), (HF, True, False)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,groups", [(1, 1, 1), (1, 300, 9), (2, 16, 2), (5, 37, 5), (16, 64, 17), (17, 65, 3), (33, 129, 4),
                                        (64, 20, 40), (65, 130, 6), (200, 50, 3)])
def test_product(M, N, groups, group, dtype, zero, bias):
    _check(M, N, groups * group, group, zero, dtype, bias)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_product_large(dtype):
    _check(1, 4099, 4096, 128, True, dtype, True)
    _check(16, 1000, 8192, 64, False, dtype, False)


def _check_grouped(counts, N, K, group, zero, dtype, bias, gather, tail):
    E, R = len(counts), sum(counts) + tail
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32)
    g = torch.Generator().manual_seed(N)
    rows = torch.randint(0, gather, (R,), generator=g).to(torch.int32) if gather else None
    if rows is not None and tail:
        rows[R - tail:] = -1
    q, s, z = pg.quantize_w4(_rand(1, E, N, K, dtype=dtype, scale=K ** -0.5).cuda(), group, zero=zero)
    x = _rand(2, gather or R, K, dtype=dtype)
    b = _rand(3, E, N, dtype=dtype) if bias else None
    put = lambda t: None if t is None else t.cuda()      # noqa: E731
    got = pg.gemm_w4(put(x), q, s, z, put(b), offsets=put(offsets), rows=put(rows))
    xs = x if rows is None else x[rows.long().clamp(min=0)]
    for e, lo, hi in ref.spans(offsets, R):
        if lo < hi:
            want, mag = ref.w4(xs[lo:hi], q[e], s[e], None if z is None else z[e], None if b is None else b[e], group)
            bound = ref.rounding(want, dtype) * 1.001 + mag * (2 * group + K // group + 8) * ref.STEP32
            ref.assert_near(got[lo:hi], want, bound, f"expert {e}")
    assert not got[sum(counts):].any()
    out = torch.full((R, N), 7.0, dtype=dtype, device="cuda")
    pg.gemm_w4(put(x), q, s, z, put(b), offsets=put(offsets), rows=put(rows), out=out)
    assert torch.equal(out[:sum(counts)], got[:sum(counts)]) and bool((out[sum(counts):] == 7.0).all())


@pytest.mark.parametrize("dtype,zero,bias,gather,tail", [(BF, False, False, 0, 0), (BF, True, True, 9, 2), (HF, True, False, 3, 0),
                                                         (HF, False, True, 0, 5)])
@pytest.mark.parametrize("counts,N,K,group", [([1], 5, 32, 32), ([0, 2, 0, 1], 40, 128, 128), ([3, 17, 0, 70], 100, 192, 64),
                                              ([16, 16], 33, 1056, 32), ([0, 0, 0, 1, 0, 0, 1, 0], 64, 512, 128)])
def test_product_by_expert(counts, N, K, group, dtype, zero, bias, gather, tail):
    _check_grouped(counts, N, K, group, zero, dtype, bias, gather, tail)


def test_product_of_values_that_are_not_finite():
    q, s, z = pg.quantize_w4(_rand(1, 64, 256, dtype=BF).cuda(), 64)
    x = _rand(2, 5, 256, dtype=BF)
    x[1, 200], x[3, 3] = math.inf, math.nan
    got = pg.gemm_w4(x.cuda(), q, s, z)
    clean = x.clone()
    clean[1], clean[3] = 0, 0
    assert bool(torch.isnan(got[[1, 3]]).all())
    want, mag = ref.w4(clean[[0, 2, 4]], q, s, z, None, 64)
    ref.assert_near(got[[0, 2, 4]], want, ref.rounding(want, BF) * 1.001 + mag * 140 * ref.STEP32)
    s[1, 7] = math.nan                       # a group's scale: its row of the weight only
    got = pg.gemm_w4(clean.cuda(), q, s, z)
    assert bool(torch.isnan(got[:, 7]).all()) and int(torch.isnan(got).sum()) == 5
