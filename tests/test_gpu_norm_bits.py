"""The norms' outputs to the last bit, given the statistics they return: the formula's products and sum one by one, each
rounded to fp32, and one rounding to the output type."""

from __future__ import annotations

import pytest
import torch

import persistent_gemm_amd as pg
from test_gpu_norm import EPS, TYPES, _case, _cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(3, 7), (40, 100), (700, 513), (5, 2047), (600, 2048), (50, 4096), (33, 8192), (9, 20001)])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("gate,scaled", [(None, False), ("vector", True), ("token", True), ("group", False)])
def test_outputs_are_the_formula_s_operations(T, D, t, gate, scaled):
    x = _cuda(_case(T, D, t, gate, scaled, T + D + 5))
    out, rstd, y, rn = pg.gated_norm(x["h"], x["residual"], x["weight"], x["gate"], x["residual_scale"], EPS,
                                     next_weight=x["next_weight"])
    n = x["h"].float() * rstd[:, None] * x["weight"].float()
    if gate:
        g = x["gate"].float().reshape(-1, D)
        n = n * g.repeat_interleave(T // g.shape[0], dim=0)
    r = x["residual"].float()
    if scaled:
        r = r * x["residual_scale"].float()
    assert torch.equal(out, (r + n).to(TYPES[t]))
    assert torch.equal(y, (out.float() * rn[:, None] * x["next_weight"].float()).to(TYPES[t]))


@pytest.mark.parametrize("D", [5, 300, 5000])
def test_mean_squares_among_the_smallest_numbers(D):
    """With eps 0 the statistic of a row of 2^-70 is 2^70: its squares are 2^-140, exactly, below the normal numbers.  A root is
    off by one step of fp32 at most, and a mean of equal squares by its rounding to multiples of 2^-149: 2^-10."""
    x = torch.full((4, D), 2.0 ** -70, device="cuda")
    x[1] = 2.0 ** -63
    x[2] = 2.0 ** 60
    x[3] = 1.0
    y, r = pg.rms_norm(x, torch.ones(D, device="cuda"), 0.0)
    want = (1 / x[:, 0].double()).cpu()
    assert ((r.double().cpu() / want - 1).abs() <= torch.tensor([2.0 ** -10, 2.0 ** -20, 2.0 ** -20, 2.0 ** -20]).double()).all()
    assert ((y.double() - 1).abs() <= 2.0 ** -9).all()
