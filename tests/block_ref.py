"""Plain 64-bit CPU forms of the block-scaled E4M3 operators and the norms, for the tests."""

from __future__ import annotations

import torch

E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -126


def up(n, m):
    return -(-n // m) * m


def pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def round_e4m3(v):
    """fp64 -> the nearest E4M3 value, ties to the even code (|v| below 464)."""
    e = torch.frexp(v).exponent.clamp(min=-5) - 4
    step = torch.ldexp(torch.ones_like(v), e)
    return torch.round(v / step) * step


def spacing(v):
    """Distance between the E4M3 values around |v|."""
    e = torch.frexp(v).exponent.clamp(min=-5) - 4
    return torch.ldexp(torch.ones_like(v), e)


def scale_of(amax):
    s = (amax / 448.0).float().double().clamp(min=TINY)
    return torch.where(torch.isfinite(amax), s, torch.nan)


def quantize(x, block):
    """x [R, C] -> (code values fp64 [R, C up to 16], scale fp64 as quantize_fp8_block lays it out)."""
    R, C = x.shape
    n = 128 if block == "tile" else 1
    p = pad(x.double().cpu(), up(R, n), up(C, 128)).reshape(up(R, n) // n, n, -1, 128)
    s = scale_of(p.abs().amax(dim=(1, 3), keepdim=True))
    q = round_e4m3(p / s).reshape(up(R, n), -1)[:R, :up(C, 16)]
    s = s[:, 0, :, 0]
    return q, (s if block == "tile" else s.t()).contiguous()


def dequantize(q, scale, block):
    """fp64 values of codes [R, Kp]."""
    R, K = q.shape
    s = scale.double().cpu()
    s = s.repeat_interleave(128, dim=0)[:R] if block == "tile" else s.t()
    return q.double().cpu() * s.repeat_interleave(128, dim=1)[:, :K]


def gate_rows(gate, T):
    if gate is None:
        return 1.0
    g = gate.double().cpu()
    g = g[None] if g.dim() == 1 else g
    return g.repeat_interleave(T // g.shape[0], dim=0)


def norm_forward(h, residual, weight, gate, residual_scale, eps):
    """(out, rstd, bound on |terms|) of the norm after a block, unrounded."""
    h, res = h.double().cpu(), residual.double().cpu()
    r = (h.square().mean(dim=1) + eps).rsqrt()
    n = h * r[:, None] * weight.double().cpu() * gate_rows(gate, h.shape[0])
    if residual_scale is not None:
        res = res * residual_scale.double().cpu()
    return res + n, r, res.abs() + n.abs()


def rms(x, weight, eps):
    x = x.double().cpu()
    r = (x.square().mean(dim=1) + eps).rsqrt()
    return x * r[:, None] * weight.double().cpu(), r


def norm_backward(dout, h, weight, rstd, gate, residual, residual_scale, dy, out, next_weight, rstd_next, sign=1.0):
    """Gradients by the formulas; with absolute inputs and sign = -1 every term counts with its magnitude,
    which bounds what roundings can add up to.  Absent parts are None."""
    d = lambda t: None if t is None else (t.double().cpu() if sign > 0 else t.double().cpu().abs())
    dout, h, weight, rstd, gate_, residual, rs, dy, out, nw, rn = map(
        d, (dout, h, weight, rstd, gate, residual, residual_scale, dy, out, next_weight, rstd_next))
    got = {}
    dv = 0.0 if dout is None else dout
    if dy is not None:
        xh = out * rn[:, None]
        got["dnext_weight"] = (dy * xh).sum(0)
        g = dy * nw
        dv = dv + rn[:, None] * (g - sign * xh * (g * xh).mean(1, keepdim=True))
    if h is None:
        got["dx"] = dv
        return got
    T, D = h.shape
    hh = h * rstd[:, None]
    dn = dv
    if gate is not None:
        g2 = gate_[None] if gate_.dim() == 1 else gate_
        dn = dv * g2.repeat_interleave(T // g2.shape[0], dim=0)
        got["dgate"] = (dv * hh * weight).reshape(g2.shape[0], -1, D).sum(1).reshape(gate_.shape)
    got["dweight"] = (dn * hh).sum(0)
    g = dn * weight
    got["dh"] = rstd[:, None] * (g - sign * hh * (g * hh).mean(1, keepdim=True))
    got["dresidual"] = dv
    if rs is not None:
        got["dresidual_scale"] = (dv * residual).sum(0)
        got["dresidual"] = dv * rs
    return got
