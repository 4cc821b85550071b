"""The operators of a layer of experts in 64 bits on the CPU, one expert and one token at a time, with the sums of
magnitudes that the tests' error bounds are made of."""

from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}     # half a step, relative
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the smallest step
STEP32 = 2.0 ** -23


def rounding(y, dtype):
    """How far a value near y may be from it after one rounding to dtype."""
    return HALF[dtype] * y.abs() + LEAST[dtype]


def assert_near(got, want, bound, what=""):
    """|got - want| <= bound everywhere; what is not finite has to be the same."""
    g, w = got.double().cpu(), want
    fine = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN in other places"
    assert torch.equal(g[~fine & ~torch.isnan(w)], w[~fine & ~torch.isnan(w)]), f"{what}: other infinities"
    d = (g - w).abs()[fine]
    b = bound.expand(w.shape)[fine] if torch.is_tensor(bound) else torch.full_like(d, bound)
    if (d > b).any():
        i = int((d / b).argmax())
        raise AssertionError(f"{what}: {int((d > b).sum())} of {d.numel()} beyond the bound, worst {d[i]:.3e} over {b[i]:.3e} "
                             f"(value {w[fine][i]:.6e})")


# ---------------------------------------------------------------- routing

def route(logits, k, normalize):
    """(experts, weights, offsets, slots, rows) of logits [T, E]."""
    x = logits.double().cpu()
    T, E = x.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        row = x[t].tolist()
        order = sorted((e for e in range(E) if row[e] > -math.inf), key=lambda e: (-row[e], e))[:k]
        if any(v != v for v in row):
            p = {e: math.nan for e in order}
        else:
            top = max(row) if E else 0.0
            ex = [0.0 if v == -math.inf else math.nan if top == math.inf else math.exp(v - top) for v in row]
            total = sum(ex[e] for e in order) if normalize else sum(ex)
            p = {e: ex[e] / total for e in order}
        for j, e in enumerate(order):
            ids[t, j], w[t, j] = e, p[e]
    return (ids, w, *places(ids, E))


def places(ids, E):
    """(offsets, slots, rows) of the choices ids [T, k]."""
    T, k = ids.shape
    by = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                by[int(ids[t, j])].append((t, j))
    offsets, slots, rows = [0], torch.full((T, k), -1, dtype=torch.int32), torch.full((T * k,), -1, dtype=torch.int32)
    for pairs in by:
        for t, j in pairs:
            rows[offsets[-1]] = t
            slots[t, j] = offsets[-1]
            offsets[-1] += 1
        offsets.append(offsets[-1])
    return torch.tensor([0] + offsets[:E], dtype=torch.int32), slots, rows


def route_weights(x, ids, normalize):
    """The weights of fixed choices, for gradients: x [T, E] double."""
    p = torch.exp(x - x.amax(dim=1, keepdim=True))
    w = p.gather(1, ids.long().clamp(min=0)) * (ids >= 0)
    return w / (w if normalize else p).sum(dim=1, keepdim=True)


def route_grad(dw, logits, ids, normalize):
    x = logits.double().cpu()
    out = torch.zeros_like(x)
    for t in range(x.shape[0]):
        at = [int(e) for e in ids[t] if e >= 0]
        if not at:
            continue
        w = route_weights(x[t:t + 1], ids[t:t + 1].cpu(), normalize)[0]
        mean = sum(float(w[j] * dw[t, j].double()) for j in range(len(at)))
        if not normalize:
            out[t] = -torch.softmax(x[t], dim=0) * mean
        for j, e in enumerate(at):
            d = float(dw[t, j])
            out[t, e] = w[j] * (d - mean)
    return out


# ---------------------------------------------------------------- products

def spans(offsets, R):
    """(expert, first row, end) of each expert, held to the rows there are."""
    o = [int(v) for v in offsets]
    out = []
    for e in range(len(o) - 1):
        a = min(max(o[e], 0), R)
        out.append((e, a, min(max(o[e + 1], a), R)))
    return out


def grouped(A, B, offsets, bias, rows):
    """(C, sums of magnitudes) with zeros behind the last expert's rows."""
    a = A.double().cpu()
    a = a if rows is None else a[rows.cpu().long().clamp(0, A.shape[0] - 1)]
    R = a.shape[0]
    C = torch.zeros(R, B.shape[1], dtype=torch.float64)
    S = torch.zeros_like(C)
    for e, lo, hi in spans(offsets, R):
        b = B[e].double().cpu()
        C[lo:hi], S[lo:hi] = a[lo:hi] @ b.t(), a[lo:hi].abs() @ b.abs().t()
        if bias is not None:
            C[lo:hi] += bias[e].double().cpu()
            S[lo:hi] += bias[e].double().cpu().abs()
    return C, S


def grouped_grad(dC, A, B, offsets, rows):
    """((dA, dB, dbias), their sums of magnitudes)."""
    a, d = A.double().cpu(), dC.double().cpu()
    a = a if rows is None else a[rows.cpu().long().clamp(0, A.shape[0] - 1)]
    R, (E, N, K) = d.shape[0], B.shape
    out = [torch.zeros(R, K, dtype=torch.float64), torch.zeros(E, N, K, dtype=torch.float64), torch.zeros(E, N, dtype=torch.float64)]
    mag = [torch.zeros_like(x) for x in out]
    for e, lo, hi in spans(offsets, R):
        b, x, g = B[e].double().cpu(), a[lo:hi], d[lo:hi]
        out[0][lo:hi], mag[0][lo:hi] = g @ b, g.abs() @ b.abs()
        out[1][e], mag[1][e] = g.t() @ x, g.abs().t() @ x.abs()
        out[2][e], mag[2][e] = g.sum(dim=0), g.abs().sum(dim=0)
    return out, mag


def combine(y, slots, weights):
    v, R = y.double().cpu(), y.shape[0]
    T, k = slots.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for t in range(T):
        for j in range(k):
            s = int(slots[t, j])
            if 0 <= s < R:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * v[s]
                mag[t] += (w * v[s]).abs()
    return out, mag


def combine_grad(dout, y, slots, weights):
    d, v, R = dout.double().cpu(), y.double().cpu(), y.shape[0]
    T, k = slots.shape
    dy, dw, mag = torch.zeros_like(v), torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            s = int(slots[t, j])
            if 0 <= s < R:
                dy[s] = (1.0 if weights is None else float(weights[t, j])) * d[t]
                dw[t, j], mag[t, j] = (d[t] * v[s]).sum(), (d[t] * v[s]).abs().sum()
    return dy, dw, mag


# ---------------------------------------------------------------- 4-bit weights

def quantize(w, group, zero, dtype):
    """(codes [N, K], scale [K / group, N] of dtype, zero points) of w [N, K].  A scale is the fp32 quotient, rounded."""
    x = w.float().cpu()
    N, K = x.shape
    least = torch.finfo(dtype).tiny
    codes = torch.zeros(N, K, dtype=torch.uint8)
    scale, zeros = torch.zeros(K // group, N, dtype=dtype), torch.full((K // group, N), 8, dtype=torch.uint8)
    for g in range(K // group):
        part = x[:, g * group:(g + 1) * group]
        bad = ~torch.isfinite(part).all(dim=1)
        part = torch.where(bad[:, None], 0.0, part)
        lo, hi = part.amin(dim=1).clamp(max=0), part.amax(dim=1).clamp(min=0)
        s = (((hi - lo) / 15) if zero else part.abs().amax(dim=1) / 7).to(dtype)
        bad |= torch.isinf(s)
        s = torch.where(torch.isinf(s), torch.ones_like(s), s).clamp(min=least)
        sd = s.double()
        z = torch.round(-lo.double() / sd).clamp(0, 15) if zero else torch.full((N,), 8.0, dtype=torch.float64)
        q = (torch.round(part.double() / sd[:, None]) + z[:, None]).clamp(0, 15)
        codes[:, g * group:(g + 1) * group] = torch.where(bad[:, None], 0.0, q).to(torch.uint8)
        scale[g] = torch.where(bad, torch.full_like(s, math.nan), s)
        zeros[g] = torch.where(bad, torch.zeros_like(z) if zero else z, z).to(torch.uint8)
    return codes, scale, zeros


def unpack(q):
    """Codes [..., K] of packed ones [..., K / 2]."""
    q = q.cpu()
    return torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)


def by_element(x, group):
    """[K / group, N] -> [N, K]."""
    return x.double().cpu().repeat_interleave(group, dim=0).t()


def w4(x, q, scale, zero, bias, group):
    """(C, the magnitudes that the kernel's form adds up) of one weight: (16 + code) x less (16 + zero) x."""
    a, c, s = x.double().cpu(), unpack(q).double(), by_element(scale, group)
    z = torch.full_like(s, 8.0) if zero is None else by_element(zero, group)
    C = a @ (s * (c - z)).t()
    S = a.abs() @ (s.abs() * (32 + c + z)).t()
    if bias is not None:
        C, S = C + bias.double().cpu(), S + bias.double().cpu().abs()
    return C, S
