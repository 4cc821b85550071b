"""4-bit weights at the ends of their types' ranges: scales of groups that span more than the largest number, and
products of rows of the largest and the smallest elements."""

from __future__ import annotations

import pytest
import torch

import experts_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _rand(seed, *shape, dtype=FP, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_groups_that_span_more_than_the_largest_number(dtype, group):
    """With zero points a finite group has the formula's scale, though max - min itself may be beyond the type."""
    big = torch.finfo(dtype).max
    w = _rand(1, 40, 3 * group).clamp(-3, 3) * (big / 4)
    w[0, 0], w[0, 1] = big, -big
    w[1, 0], w[1, 1] = 0.59 * big, -0.59 * big
    w[2, 0], w[2, 1] = big, -0.01 * big
    w[3, 0], w[3, 1] = 0.01 * big, -big
    w[4], w[5] = w[4].abs(), -w[5].abs()
    w[6] = _rand(2, 3 * group) * 0.02            # (an ordinary row beside them)
    w = w.clamp(-big, big).to(dtype)
    q, s, z = (t.cpu() for t in pg.quantize_w4(w.cuda(), group, zero=True))
    codes = ref.unpack(q).double()
    for g in range(3):
        part = w[:, g * group:(g + 1) * group].double()
        lo, hi = part.amin(dim=1).clamp(max=0), part.amax(dim=1).clamp(min=0)
        want = (hi - lo) / 15
        # the difference and the quotient are rounded to fp32, and the scale to its type
        assert bool(((s[g].double() - want).abs() <= ref.rounding(want, s.dtype) * (1 + 2.0 ** -12) + want * 2 * 2.0 ** -24).all())
        sd = s[g].double()
        zero = torch.round(-lo / sd).clamp(0, 15)
        assert torch.equal(z[g].double(), zero)
        assert torch.equal(codes[:, g * group:(g + 1) * group], (torch.round(part / sd[:, None]) + zero[:, None]).clamp(0, 15))


def _near(got, x, q, s, z, b, group):
    want, mag = ref.w4(x, q, s, z, b, group)
    K = x.shape[1]
    assert bool((want.abs() < torch.finfo(x.dtype).max).all())
    # each addition in fp32 is off by at most a step; bf16's sums are 2^-12 of the formula's, so that half the smallest step of fp32
    # is 2^-138 there: times a scale, for each of 2 K terms, and once for each group
    least = (2 * K * float(s.double().abs().max()) + K // group + 8) * 2.0 ** -138
    ref.assert_near(got, want, ref.rounding(want, x.dtype) * 1.001 + mag * (2 * group + K // group + 8) * ref.STEP32 + least)


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,N,K", [(1, 40, 128), (3, 37, 384), (6, 64, 512), (40, 36, 256)])
def test_product_of_the_largest_and_smallest_elements(M, N, K, group, dtype, zero):
    """Finite rows have finite products where the formula has, and rows of the smallest numbers are not lost."""
    f = torch.finfo(dtype)
    w = _rand(M, 3, N, K, dtype=dtype, scale=1e-3)
    q, s, z = pg.quantize_w4(w.cuda(), group, zero=zero)
    x = _rand(1, M, K).clamp(-4, 4) * (f.max / 4)
    x[0] = f.max
    o = torch.tensor([0, M // 2, M // 2, M], dtype=torch.int32)
    for x in (x.clamp(-f.max, f.max).to(dtype), (_rand(2, M, K) * f.tiny).to(dtype)):
        one = lambda e: (q[e], s[e], None if z is None else z[e])       # noqa: E731
        _near(pg.gemm_w4(x.cuda(), *one(1)), x, *one(1), None, group)
        got = pg.gemm_w4(x.cuda(), q, s, z, offsets=o.cuda())
        for e, lo, hi in ref.spans(o, M):
            if lo < hi:
                _near(got[lo:hi], x[lo:hi], *one(e), None, group)
