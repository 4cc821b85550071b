"""The norms' backward with many rows of the gate: a worker then takes several of them.

Tolerances as in test_gpu_norm.py."""

from __future__ import annotations

import pytest
import torch

import block_ref as ref
import persistent_gemm_amd as pg
from test_gpu_norm import EPS, TYPES, _case, _check_grads, _cuda, _grads

pytestmark = pytest.mark.gpu


def _with_gates(T, D, G, t, scaled):
    x = _case(T, D, t, "token", scaled, T + D + G)
    x["gate"] = x["gate"][:G].contiguous()
    return x


# (workers of a wave: 2048 at once; of 256, 512 and 1024 threads: 512, 256 and 128; the last worker's share whole or not)
@pytest.mark.parametrize("T,D,G", [(5000, 100, 2500), (6150, 300, 2050), (1200, 700, 600), (1030, 1001, 515), (600, 2500, 300),
                                   (514, 4095, 257), (780, 2304, 260), (600, 5000, 300), (520, 8192, 260), (274, 9000, 137),
                                   (270, 17000, 135)])
@pytest.mark.parametrize("t,scaled,pre", [("bf16", True, True), ("fp32", False, False), ("fp32", True, True)])
def test_more_gate_rows_than_workers(T, D, G, t, scaled, pre):
    x = _with_gates(T, D, G, t, scaled)
    d = _cuda(x)
    fwd = pg.gated_norm(d["h"], d["residual"], d["weight"], d["gate"], d["residual_scale"], EPS,
                        next_weight=d["next_weight"] if pre else None)
    out, rstd, rn = fwd[0], fwd[1], fwd[3] if pre else None
    nxt = dict(dy=d["dy"], out=out, next_weight=d["next_weight"], rstd_next=rn) if pre else {}
    call = lambda: dict(zip(("dh", "dresidual", "dweight", "dgate", "dresidual_scale", "dnext_weight"),
                            pg.gated_norm_backward(d["dout"], d["h"], d["weight"], rstd, d["gate"], d["residual"],
                                                   d["residual_scale"], **nxt)))
    got = call()
    want, bound = _grads(x, rstd, rn, out, pre), _grads(x, rstd, rn, out, pre, sign=-1.0)
    assert {k for k, v in got.items() if v is not None} == set(want)
    _check_grads(got, want, bound, T, t, f"{T}x{D} {G} {t}")
    again = call()
    assert all(v is None or torch.equal(v, again[k]) for k, v in got.items())


@pytest.mark.parametrize("T,D,G", [(8192, 8192, 4096), (8192, 512, 4096), (4096, 2048, 2048)])
def test_scratch_does_not_grow_with_the_gate(T, D, G):
    """Three rows of fp32 sums for each worker that runs at once (512 threads to a compute unit, 64 or more a
    worker), and what the allocator rounds up."""
    x = torch.randn(T, D, device="cuda").to(torch.bfloat16)
    w, gate, r = x[0].clone(), x[:G].clone(), torch.ones(T, device="cuda")
    args = dict(residual=x, residual_scale=w, dy=x, out=x, next_weight=w, rstd_next=r)
    pg.gated_norm_backward(x, x, w, r, gate, **args)
    torch.cuda.synchronize()
    pg.release_workspace()
    free = torch.cuda.mem_get_info()[0]
    pg.gated_norm_backward(x, x, w, r, gate, **args)
    torch.cuda.synchronize()
    took = free - torch.cuda.mem_get_info()[0]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    threads = 64 if D <= 512 else 256 if D <= 2048 else 512
    assert took <= 3 * 4 * D * (512 * cus // threads) + (4 << 20), took
