"""The norms before and after a block on the GPU, forward and backward, against 64-bit forms on the CPU.

Tolerances count roundings.  A mean over a row is a chain of at most 32 additions in a thread and 10 across
threads (and 16 more between waves): below 60 steps of 2^-24; a root halves what its argument is off by.  What is
stored is off by half a step more.  For the gradients every term is counted with its magnitude (`bound`): two means in a
row and about 40 other operations are below 200 steps, and a column sum over T rows adds at most T + 60."""

from __future__ import annotations

import pytest
import torch

import block_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
EPS = 1e-6

# rows of one wave, of 256 and 1024 threads, of one and several pieces a thread; odd ones; the widest
SHAPES = [(1, 1), (3, 7), (5, 64), (9, 130), (600, 511), (5, 512), (7, 1000), (530, 1001), (4, 2047), (520, 2048),
          (3, 4096), (515, 4095), (2, 8190), (513, 8192), (2, 20001), (1, 32768)]


def _half(t):
    return torch.finfo(t).eps / 2


def _case(T, D, t, gate, scaled, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    x = dict(h=r(T, D) * torch.exp(r(T, 1)), residual=2 * r(T, D), weight=1 + 0.1 * r(D), next_weight=1 + 0.1 * r(D),
             gate=None, residual_scale=1 + 0.1 * r(D) if scaled else None, dout=r(T, D), dy=r(T, D))
    if gate:
        G = {"vector": None, "one": 1, "token": T, "group": next(n for n in (4, 3, 2, 1) if T % n == 0)}[gate]
        x["gate"] = 0.5 + 0.2 * (r(D) if G is None else r(G, D))
    return {k: None if v is None else v.to(TYPES[t]) for k, v in x.items()}


def _cuda(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def _close(got, want, tol, what):
    err = (got.double().cpu() - want).abs() - tol
    assert (err <= 0).all(), f"{what}: off by {err.max().item()} more than allowed"


def _check_codes(q, s, y, rel, what):
    """Codes and scales against y (fp64), which the kernel has within `rel`."""
    T, D = y.shape
    blocks = ref.up(D, 128) // 128
    _, ws = ref.quantize(y.float(), "row")
    assert ((s.double().cpu() - ws).abs() <= ws * (rel + 2 * U)).all(), what
    got = q.cpu().float().double()
    assert got.shape == (T, ref.up(D, 16)) and s.shape == (blocks, T)
    assert (got[:, D:] == 0).all(), what
    v = y / s.double().cpu().t().repeat_interleave(128, dim=1)[:, :D]
    assert ((got[:, :D] - v).abs() <= ref.spacing(v.abs() * (1 + rel)) / 2 + v.abs() * (rel + U)).all(), what


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_rms_norm(T, D, t):
    x = _case(T, D, t, None, False, T + D)
    d = _cuda(x)
    want, r = ref.rms(x["h"], x["weight"], EPS)
    y, rstd = pg.rms_norm(d["h"], d["weight"], EPS)
    _close(rstd, r, 33 * U * r, "rstd")
    _close(y, want, want.abs() * (40 * U + _half(TYPES[t])), "y")
    q, s, rstd2 = pg.rms_norm(d["h"], d["weight"], EPS, quantize=True)
    assert torch.equal(rstd, rstd2)
    _check_codes(q, s, want, 40 * U, f"codes {T}x{D} {t}")


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("gate,scaled", [(None, False), ("vector", True), ("token", False), ("group", True)])
def test_gated_norm(T, D, t, gate, scaled):
    x = _case(T, D, t, gate, scaled, T + D)
    d = _cuda(x)
    args = (d["h"], d["residual"], d["weight"], d["gate"], d["residual_scale"], EPS)
    want, r, bound = ref.norm_forward(x["h"], x["residual"], x["weight"], x["gate"], x["residual_scale"], EPS)
    out, rstd = pg.gated_norm(*args)
    _close(rstd, r, 33 * U * r, "rstd")
    _close(out, want, bound * 40 * U + want.abs() * _half(TYPES[t]) + bound * 40 * U * _half(TYPES[t]), "out")
    out2, rstd2, y, rn = pg.gated_norm(*args, next_weight=d["next_weight"])
    assert torch.equal(out, out2) and torch.equal(rstd, rstd2)
    want, r = ref.rms(out, x["next_weight"], EPS)     # of what was stored
    _close(rn, r, 33 * U * r, "rstd_next")
    _close(y, want, want.abs() * (40 * U + _half(TYPES[t])), "y")
    out3, rstd3, q, s, rn3 = pg.gated_norm(*args, next_weight=d["next_weight"], quantize=True)
    assert torch.equal(out, out3) and torch.equal(rstd, rstd3) and torch.equal(rn, rn3)
    _check_codes(q, s, want, 40 * U, f"codes {T}x{D} {t}")


def _grads(x, rstd, rstd_next, out, pre, sign=1.0):
    nxt = (x["dy"], out, x["next_weight"], rstd_next) if pre else (None,) * 4
    return ref.norm_backward(x["dout"], x["h"], x["weight"], rstd, x["gate"], x["residual"], x["residual_scale"], *nxt,
                             sign=sign)


def _check_grads(got, want, bound, T, t, what):
    for k, w in want.items():
        steps = 200 + (T + 60 if w.dim() == 1 or k == "dgate" else 0)
        tol = bound[k] * steps * U + w.abs() * _half(TYPES[t]) + 2.0 ** -133
        _close(got[k], w, tol, f"{what}: {k}")


@pytest.mark.parametrize("T,D", SHAPES + [(2000, 200), (2050, 640)])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("gate,scaled,pre", [(None, False, False), ("vector", True, True), ("token", False, True),
                                             ("group", True, False), ("one", False, True)])
def test_gated_norm_backward(T, D, t, gate, scaled, pre):
    x = _case(T, D, t, gate, scaled, T + D)
    d = _cuda(x)
    fwd = pg.gated_norm(d["h"], d["residual"], d["weight"], d["gate"], d["residual_scale"], EPS,
                        next_weight=d["next_weight"] if pre else None)
    out, rstd = fwd[:2]
    nxt = dict(dy=d["dy"], out=out, next_weight=d["next_weight"], rstd_next=fwd[3]) if pre else {}
    call = lambda: dict(zip(("dh", "dresidual", "dweight", "dgate", "dresidual_scale", "dnext_weight"),
                            pg.gated_norm_backward(d["dout"], d["h"], d["weight"], rstd, d["gate"], d["residual"],
                                                   d["residual_scale"], **nxt)))
    got = call()
    want = _grads(x, rstd, fwd[3] if pre else None, out, pre)
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k, w in want.items():
        assert got[k].shape == w.shape and got[k].dtype == TYPES[t], k
    bound = _grads(x, rstd, fwd[3] if pre else None, out, pre, sign=-1.0)
    _check_grads(got, want, bound, T, t, f"{T}x{D} {t} {gate}")
    again = call()
    assert all(v is None or torch.equal(v, again[k]) for k, v in got.items())


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_rms_norm_backward(T, D, t):
    x = _case(T, D, t, None, False, T + D + 1)
    d = _cuda(x)
    _, rstd = pg.rms_norm(d["h"], d["weight"], EPS)
    for extra in (None, "dout"):
        dx, dw = pg.rms_norm_backward(d["dy"], d["h"], d["weight"], rstd, d[extra] if extra else None)
        args = (x[extra] if extra else None, None, None, None, None, None, None, x["dy"], x["h"], x["weight"], rstd)
        want, bound = ref.norm_backward(*args), ref.norm_backward(*args, sign=-1.0)
        _check_grads({"dx": dx, "dnext_weight": dw}, want, bound, T, t, f"{T}x{D} {t} {extra}")


def test_gradients_against_differences():
    """The kernel's fp32 gradients against central differences of the 64-bit forward, both norms in a chain."""
    T, D = 6, 40
    x = _case(T, D, "fp32", "group", True, 77)
    d = _cuda(x)
    out, rstd, y, rn = pg.gated_norm(d["h"], d["residual"], d["weight"], d["gate"], d["residual_scale"], EPS,
                                     next_weight=d["next_weight"])
    got = dict(zip(("h", "residual", "weight", "gate", "residual_scale", "next_weight"),
                   pg.gated_norm_backward(d["dout"], d["h"], d["weight"], rstd, d["gate"], d["residual"],
                                          d["residual_scale"], dy=d["dy"], out=out, next_weight=d["next_weight"],
                                          rstd_next=rn)))

    def loss(z):
        o, _, _ = ref.norm_forward(z["h"], z["residual"], z["weight"], z["gate"], z["residual_scale"], EPS)
        n, _ = ref.rms(o, z["next_weight"], EPS)
        return (o * z["dout"]).sum() + (n * z["dy"]).sum()

    z = {k: v.double() for k, v in x.items()}
    g = torch.Generator().manual_seed(1)
    for name, grad in got.items():
        u = torch.randn(z[name].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        diff = (loss({**z, name: z[name] + step * u}) - loss({**z, name: z[name] - step * u})) / (2 * step)
        along = (grad.double().cpu() * u).sum()
        # fp32 gradients of order 1 (a few 2^-24 each, some hundred of them) and the differences' own 1e-10 / 1e-5
        assert abs(diff - along) <= 1e-4 * (1 + (grad.double().cpu() * u).abs().sum()), name


def test_zero_rows_and_special_values():
    for t in TYPES.values():
        x = torch.randn(5, 256).to(t).cuda()
        w = torch.ones(256, dtype=t, device="cuda")
        x[1] = 0
        x[3, 7] = float("nan")
        x[4, 9] = float("inf")
        y, r = pg.rms_norm(x, w)
        q, s, _ = pg.rms_norm(x, w, quantize=True)
        assert torch.equal(y[1], torch.zeros_like(y[1])) and abs(r[1].item() - 1000.0) < 0.01
        assert (s[:, 1] == 2.0 ** -126).all() and (q[1].view(torch.uint8) == 0).all()
        assert y[3].isnan().all() and s[:, 3].isnan().all() and q[3].float().isnan().all()
        assert y[4, 9].isnan() and (y[4, :9] == 0).all()
        assert torch.isfinite(y[0].float()).all() and torch.isfinite(y[2].float()).all()


def test_out_may_take_an_input_s_place():
    """The C entry lets out be h or residual itself."""
    import ctypes
    T, D = 300, 1000
    x = _cuda(_case(T, D, "bf16", "token", True, 5))
    want, rstd = pg.gated_norm(x["h"], x["residual"], x["weight"], x["gate"], x["residual_scale"], EPS)
    for name in ("h", "residual"):
        z = dict(x, **{name: x[name].clone()})
        r = torch.empty_like(rstd)
        a = pg._NormArgs(elem=0, eps=EPS, T=T, D=D, gates=T, out=z[name].data_ptr(), rstd=r.data_ptr(),
                         stream=torch.cuda.current_stream().cuda_stream,
                         **{k: z[k].data_ptr() for k in ("h", "residual", "weight", "gate", "residual_scale")})
        assert pg.load().sk_norm_forward(ctypes.byref(a)) == 0
        assert torch.equal(z[name], want) and torch.equal(r, rstd)


def test_offsets_past_32_bits():
    T, D = 70000, 32000
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.randn(5, D, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q, s, r = pg.rms_norm(x, w, quantize=True)
    q2, s2, r2 = pg.rms_norm(x[-5:].contiguous(), w, quantize=True)
    assert torch.equal(q[-5:].view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s[:, -5:], s2) and torch.equal(r[-5:], r2)
    del q, s
    dx, dw = pg.rms_norm_backward(x, x, w, r)
    dx2, dw2 = pg.rms_norm_backward(x[-5:].contiguous(), x[-5:].contiguous(), w, r2)
    assert torch.equal(dx[-5:], dx2) and (dx[:-5] == 0).all()
    assert torch.allclose(dw.float(), dw2.float(), rtol=2.0 ** -7, atol=1e-6)


def test_views_that_start_anywhere():
    flat = torch.randn(3 + 20 * 96).to(torch.bfloat16).cuda()
    x, w = flat[3:].view(20, 96), flat[1:97]
    y, r = pg.rms_norm(x, w)
    y2, r2 = pg.rms_norm(x.clone(), w.clone())
    assert torch.equal(y, y2) and torch.equal(r, r2)


def test_forward_replays_in_a_graph_and_backward_refuses():
    x = _cuda(_case(100, 512, "bf16", "token", True, 9))
    call = lambda: pg.gated_norm(x["h"], x["residual"], x["weight"], x["gate"], x["residual_scale"], EPS,
                                 next_weight=x["next_weight"], quantize=True)
    _, rstd = call()[:2]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
        with pytest.raises(pg.SkError, match="UNSUPPORTED"):
            pg.rms_norm_backward(x["dy"], x["h"], x["weight"], rstd)
    for k in range(4):
        x["h"].copy_(torch.randn(100, 512, generator=torch.Generator().manual_seed(k)).to(torch.bfloat16))
        eager = call()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, eager)), k


def test_refusals():
    x = _cuda(_case(6, 64, "bf16", "token", True, 10))
    h, res, w, r = x["h"], x["residual"], x["weight"], torch.ones(6, device="cuda")
    for bad, kind in ((lambda: pg.rms_norm(h.half(), w), TypeError),
                      (lambda: pg.rms_norm(h, w.float()), TypeError),
                      (lambda: pg.rms_norm(h, w[:5]), ValueError),
                      (lambda: pg.rms_norm(h.t(), w), ValueError),
                      (lambda: pg.rms_norm(h[:0], w), pg.SkError),
                      (lambda: pg.rms_norm(torch.zeros(1, 32769, device="cuda"), torch.zeros(32769, device="cuda")),
                       pg.SkError),
                      (lambda: pg.gated_norm(h, res, w, x["gate"][:4]), ValueError),
                      (lambda: pg.gated_norm(h, res[:3], w), ValueError),
                      (lambda: pg.gated_norm(h, res, w, quantize=True), ValueError),
                      (lambda: pg.gated_norm_backward(h, h, w, r, residual_scale=w), TypeError),
                      (lambda: pg.gated_norm_backward(h, h, w, r, dy=h), TypeError),
                      (lambda: pg.gated_norm_backward(h, h, w, r, out=h), ValueError),
                      (lambda: pg.rms_norm_backward(h, h, w, r.double()), TypeError)):
        with pytest.raises(kind):
            bad()
