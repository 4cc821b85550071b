"""Products by expert with 4-bit weights, few rows to an expert on the average and many to some: parts of K that LDS holds one after
the other, and several turns of rows, in the kernels that aligned weights of few rows take."""

from __future__ import annotations

import pytest
import torch

import experts_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _rand(seed, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


@pytest.mark.parametrize("dtype,zero,bias,gather", [(BF, False, True, 0), (BF, True, False, 11), (HF, False, False, 11), (HF, True, True, 0)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts,N,K", [
    ([6, 1, 0, 16, 3, 0, 2, 1], 100, 4096), ([0, 40, 0, 1, 0, 0, 2, 0], 68, 2048), ([0, 40, 0, 1, 0, 0, 2, 0], 36, 2176),
    ([17, 33, 0, 1, 0, 0, 0, 0], 32, 1152), ([0] * 63 + [100], 20, 640),
])
def test_skewed_loads(counts, N, K, group, dtype, zero, bias, gather):
    E, R = len(counts), sum(counts)
    assert -(-R // E) <= 8 and N % 4 == 0
    offsets = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32)
    rows = torch.randint(0, gather, (R,), generator=torch.Generator().manual_seed(N)).to(torch.int32) if gather else None
    q, s, z = pg.quantize_w4(_rand(1, E, N, K, dtype=dtype, scale=K ** -0.5).cuda(), group, zero=zero)
    x = _rand(2, gather or R, K, dtype=dtype)
    b = _rand(3, E, N, dtype=dtype) if bias else None
    put = lambda t: None if t is None else t.cuda()      # noqa: E731
    got = pg.gemm_w4(put(x), q, s, z, put(b), offsets=put(offsets), rows=put(rows))
    xs = x if rows is None else x[rows.long()]
    for e, lo, hi in ref.spans(offsets, R):
        if lo < hi:
            want, mag = ref.w4(xs[lo:hi], q[e], s[e], None if z is None else z[e], None if b is None else b[e], group)
            # 2 K terms, K / group products with a scale, eight sums of waves and the bias, each addition off by at most a step
            ref.assert_near(got[lo:hi], want, ref.rounding(want, dtype) * 1.001 + mag * (2 * group + K // group + 8) * ref.STEP32, f"expert {e}")
    again = pg.gemm_w4(put(x), q, s, z, put(b), offsets=put(offsets), rows=put(rows))
    assert torch.equal(got, again)
