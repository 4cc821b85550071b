"""Argument checks of the block-scaled and norm entry points of the C ABI (no GPU: they come before any device
work), and the 64-bit gradient forms of the tests against differences."""

from __future__ import annotations

import ctypes

import pytest
import torch

import block_ref as ref
import persistent_gemm_amd as pg

X, Q, S, QT, ST = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000


@pytest.mark.parametrize("args,status", [
    ((None, 0, 0, Q, S, None, None, 8, 8), 1), ((X, 2, 0, Q, S, None, None, 8, 8), 1),
    ((X, 0, 2, Q, S, None, None, 8, 8), 1), ((X, 0, 0, None, None, None, None, 8, 8), 1),
    ((X, 0, 0, Q, None, None, None, 8, 8), 1), ((X, 0, 0, Q, S, QT, None, 8, 8), 1),
    ((X, 0, 0, Q, S, None, None, 0, 8), 1), ((X, 0, 0, Q, S, None, None, 8, 1 << 31), 1),
    ((X, 0, 0, Q, S, None, None, 1 << 30, 1 << 30), 1),
    ((X + 1, 0, 0, Q, S, None, None, 8, 8), 2), ((X + 2, 1, 0, Q, S, None, None, 8, 8), 2),
    ((X, 0, 0, Q + 8, S, None, None, 8, 8), 2), ((X, 0, 0, Q, S + 2, None, None, 8, 8), 2),
    ((X, 0, 0, X + 32, S, None, None, 8, 8), 1),          # codes over x
    ((X, 0, 0, Q, S, Q + 16, ST, 8, 8), 1),               # both forms' codes over each other
])
def test_quantize_checks(args, status):
    assert pg.load().sk_quantize_fp8_block(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(A=None), 1), (dict(SA=None), 1), (dict(SB=None), 1), (dict(C=None), 1), (dict(block=2), 1),
    (dict(M=0), 1), (dict(N=(1 << 22) + 1), 1), (dict(K=(1 << 21) + 16), 1), (dict(M=1 << 31), 1),
    (dict(K=24), 2), (dict(A=X + 8), 2), (dict(C=0x600008), 2), (dict(SA=S + 2), 2), (dict(bias=0x700001), 2),
    (dict(C=X + 64), 1), (dict(bias=0x600000), 1),
])
def test_gemm_checks(kw, status):
    a = dict(A=X, B=Q, SA=S, SB=ST, block=1, bias=None, C=0x600000, M=64, N=64, K=128)
    a.update(kw)
    assert pg.load().sk_gemm_fp8_block(a["A"], a["B"], a["SA"], a["SB"], a["block"], a["bias"], a["C"], a["M"], a["N"],
                                       a["K"], 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dC=None), 1), (dict(dA=None, dB=None, db=None), 1), (dict(At=None), 1), (dict(Bt_s=None), 1),
    (dict(M=0), 1), (dict(K=(1 << 22) + 1), 1), (dict(N=(1 << 21) + 1), 1),
    (dict(dC=X + 1), 2), (dict(dA=0x600008), 2), (dict(At_s=S + 1), 2),
    (dict(dA=X), 1), (dict(dB=0x600010), 1), (dict(db=0x700000), 1),
])
def test_gemm_backward_checks(kw, status):
    a = dict(dC=X, At=Q, At_s=S, Bt=QT, Bt_s=ST, dA=0x600000, dB=0x700000, db=0x800000, M=64, N=64, K=64)
    a.update(kw)
    assert pg.load().sk_gemm_fp8_block_backward(a["dC"], a["At"], a["At_s"], a["Bt"], a["Bt_s"], a["dA"], a["dB"],
                                                a["db"], a["M"], a["N"], a["K"], 0, None) == status


FWD = dict(elem=0, eps=1e-6, h=0x100000, residual=0x200000, weight=0x300000, out=0x400000, rstd=0x500000, T=8, D=64)
PRE = dict(next_weight=0x600000, y=0x700000, rstd_next=0x800000)


@pytest.mark.parametrize("kw,status", [
    (dict(elem=2), 1), (dict(residual=None), 1), (dict(weight=None), 1), (dict(out=None), 1), (dict(rstd=None), 1),
    (dict(h=None), 1), (dict(T=0), 1), (dict(D=0), 1), (dict(D=32769), 1), (dict(T=1 << 31), 1),
    (dict(gate=0x900000), 1), (dict(gate=0x900000, gates=3), 1), (dict(gate=0x900000, gates=9), 1), (dict(gates=1), 1),
    (dict(y=0x700000), 1), (dict(next_weight=0x600000), 1), (dict(PRE, y=None), 1), (dict(PRE, q=0x900000), 1),
    (dict(PRE, q=0x900000, scale=0xA00000), 1), (dict(PRE, rstd_next=None), 1),
    (dict(h=0x100001), 2), (dict(elem=1, out=0x400002), 2), (dict(rstd=0x500001), 2),
    (dict(PRE, y=None, q=0x700008, scale=0xA00000), 2),
    (dict(out=0x100002), 1), (dict(out=0x300000), 1), (dict(rstd=0x400000), 1), (dict(PRE, y=0x200000), 1),
])
def test_norm_forward_checks(kw, status):
    a = pg._NormArgs(**{**FWD, **kw})
    assert pg.load().sk_norm_forward(ctypes.byref(a)) == status


BWD = dict(elem=0, dout=0x100000, h=0x200000, weight=0x300000, rstd=0x400000, dx=0x500000, dresidual=0x600000,
           dweight=0x700000, T=8, D=64)


@pytest.mark.parametrize("kw,status", [
    (dict(elem=-1), 1), (dict(dx=None), 1), (dict(dout=None), 1), (dict(weight=None), 1), (dict(dresidual=None), 1),
    (dict(dweight=None), 1), (dict(h=None), 1), (dict(dy=0x800000), 1), (dict(dnext_weight=0x800000), 1),
    (dict(gate=0x800000, gates=8), 1), (dict(dgate=0x800000), 1), (dict(residual_scale=0x800000), 1),
    (dict(residual_scale=0x800000, dresidual_scale=0x900000), 1), (dict(gate=0x800000, dgate=0x900000, gates=5), 1),
    (dict(T=0), 1), (dict(D=40000), 1), (dict(dout=0x100001), 2), (dict(rstd=0x400002), 2),
    (dict(dx=0x100000), 1), (dict(dresidual=0x500000), 1),
])
def test_norm_backward_checks(kw, status):
    a = pg._NormGradArgs(**{**BWD, **kw})
    assert pg.load().sk_norm_backward(ctypes.byref(a)) == status
    assert pg.load().sk_norm_backward(None) == 1 and pg.load().sk_norm_forward(None) == 1


def test_gradient_formulas_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    T, D = 6, 20
    z = dict(h=r(T, D), residual=r(T, D), weight=1 + 0.1 * r(D), gate=r(3, D), residual_scale=1 + 0.1 * r(D),
             next_weight=1 + 0.1 * r(D))
    dout, dy = r(T, D), r(T, D)

    def forward(z):
        o, a, _ = ref.norm_forward(z["h"], z["residual"], z["weight"], z["gate"], z["residual_scale"], 1e-6)
        n, b = ref.rms(o, z["next_weight"], 1e-6)
        return (o * dout).sum() + (n * dy).sum(), o, a, b

    _, o, a, b = forward(z)
    got = ref.norm_backward(dout, z["h"], z["weight"], a, z["gate"], z["residual"], z["residual_scale"], dy, o,
                            z["next_weight"], b)
    for name in z:
        u = r(*z[name].shape)
        diff = (forward({**z, name: z[name] + 1e-6 * u})[0] - forward({**z, name: z[name] - 1e-6 * u})[0]) / 2e-6
        assert abs(diff - (got["d" + name] * u).sum()) < 1e-6 * (1 + diff.abs()), name


def test_quantiser_form_against_torch():
    """The tests' E4M3 rounding against torch's cast, which rounds fp32 values to nearest-even."""
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(4)) * 100
    assert torch.equal(ref.round_e4m3(x.double()), x.to(ref.E4M3).double())
