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
