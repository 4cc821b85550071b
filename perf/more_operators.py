"""Timed cases of the operators of a layer of experts: routing, products grouped by expert, and products with
4-bit weights.

With T tokens, E experts, k experts to a token, and a pair (t, j) for the j-th expert of token t:

- ``moe_route``: the k largest logits of each token (ties to the lowest expert; an expert whose logit is -inf is never
  chosen), their weights in a softmax over the chosen ones or over all experts, and where each pair's row lies when the
  pairs are sorted by expert (in the order of the pairs within one): offsets [E + 1], slots [T, k], and the token of each
  row.  A choice that is missing has expert and slot -1 and weight 0.  ``moe_route_backward``: the logits' gradient.
- ``gemm_grouped``: C[r, n] = sum_k A[rows[r], k] B[e, n, k] + bias[e, n] for the rows r of expert e, zeros behind the
  last expert's; ``gemm_grouped_backward``: dA[r] = dC[r] B[e], dB[e] = sum_r dC[r]^T A[rows[r]], dbias[e] = sum_r dC[r].
- ``moe_combine``: out[t] = sum_j weights[t, j] y[slots[t, j]]; ``moe_combine_backward``: dy and dweights.
- ``gemm_w4``: C[m, n] = sum_k x[m, k] s[k / group, n] (q[n, k] - z[k / group, n]) + bias[n], also grouped by expert.
- ``quantize_w4`` and ``dequantize_w4``: 4-bit codes of a weight with a scale (and a zero point) for each group along a
  row, and the values they stand for.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # serving: one token chooses its experts
        {"name": "route 1 of 64", "op": "route", "T": 1, "E": 64, "k": 6, "type": "fp32", "normalize": True,
         "pad": 0.0, "backward": False},
        # a training step's routing of a batch whose last tokens are padding, with the logits' gradient
        {"name": "route 16384 of 256 with gradient", "op": "route", "T": 16384, "E": 256, "k": 8, "type": "fp32",
         "normalize": False, "pad": 0.1, "backward": True},
        # serving: a few tokens through experts of a square projection; nearly every expert's weights are read
        {"name": "grouped 4x2 of 8 4096x4096", "op": "grouped", "T": 4, "E": 8, "k": 2, "N": 4096, "K": 4096,
         "type": "bf16", "bias": False, "gather": True, "pad": 0.0},
        # a prompt of odd length through experts of odd width, with bias
        {"name": "grouped 1037x4 of 16 2051x1288", "op": "grouped", "T": 1037, "E": 16, "k": 4, "N": 2051, "K": 1288,
         "type": "fp16", "bias": True, "gather": True, "pad": 0.0},
        # a training step's forward product: the tokens are gathered as they are read
        {"name": "grouped 8192x2 of 8 4096x4096", "op": "grouped", "T": 8192, "E": 8, "k": 2, "N": 4096, "K": 4096,
         "type": "bf16", "bias": False, "gather": True, "pad": 0.0},
        # the backward of a training step's second product, whose rows lie by expert already
        {"name": "grouped backward 4001x2 of 8 2048x4096", "op": "grouped_backward", "T": 4001, "E": 8, "k": 2,
         "N": 2048, "K": 4096, "type": "bf16", "bias": True, "gather": False, "pad": 0.0},
        # the experts' outputs added up for each token
        {"name": "combine 8192x2x4096", "op": "combine", "T": 8192, "E": 8, "k": 2, "D": 4096, "type": "bf16",
         "weighted": True, "pad": 0.0, "backward": False},
        # its gradients, for a ragged batch of odd width with padding
        {"name": "combine backward 1037x4x2051", "op": "combine", "T": 1037, "E": 16, "k": 4, "D": 2051, "type": "bf16",
         "weighted": True, "pad": 0.1, "backward": True},
        # serving: one token through a wide projection with 4-bit weights
        {"name": "w4 1x8192x8192", "op": "w4", "M": 1, "N": 8192, "K": 8192, "group": 128, "zero": False,
         "type": "bf16", "bias": False},
        # serving: a decode batch through experts with 4-bit weights and zero points
        {"name": "w4 16x2 of 8 4096x4096", "op": "w4_grouped", "T": 16, "E": 8, "k": 2, "N": 4096, "K": 4096,
         "group": 64, "zero": True, "type": "fp16", "bias": True, "gather": True, "pad": 0.0},
        # a large weight made ready for serving, and read back
        {"name": "quantize 4-bit 8192x8192", "op": "quantize", "N": 8192, "K": 8192, "group": 128, "zero": False,
         "type": "bf16"},
        # the same of a weight with few rows, with zero points
        {"name": "quantize 4-bit 515x1312 zero", "op": "quantize", "N": 515, "K": 1312, "group": 32, "zero": True,
         "type": "fp32"},
    ]


def _log_size(rng, lo, hi, step=1):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 256:      # half of the larger ones are the usual multiples
        n -= n % 128
    return min(max(n - n % step, lo), hi)


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "grouped_backward", "combine", "w4", "w4_grouped", "quantize"])
    k = rng.choice([1, 2, 2, 4, 6, 8])
    E = rng.choice([8, 16, 32, 64])
    pad = rng.choice([0.0, 0.0, 0.1])
    if op == "route":
        return {"op": op, "T": _log_size(rng, 1, 16384), "E": rng.choice([5, 8, 16, 60, 64, 128, 256]), "k": min(k, 5),
                "type": rng.choice(["fp32", "bf16", "fp16"]), "normalize": rng.random() < 0.5, "pad": pad,
                "backward": rng.random() < 0.5}
    if op in ("grouped", "grouped_backward"):
        step = 8 if op == "grouped_backward" else 1
        N, K = _log_size(rng, 64, 4096, step), _log_size(rng, 64, 4096, 8)
        while E * N * K > 1 << 27:
            E //= 2
        most = 8192 if op == "grouped" else 4096
        return {"op": op, "T": _log_size(rng, 1, most // max(1, k // 2)), "E": E, "k": min(k, E), "N": N, "K": K,
                "type": rng.choice(["bf16", "bf16", "fp16"]), "bias": rng.random() < 0.5, "gather": rng.random() < 0.5,
                "pad": pad}
    if op == "combine":
        return {"op": op, "T": _log_size(rng, 1, 16384 // k), "E": E, "k": k, "D": _log_size(rng, 64, 4096),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "weighted": rng.random() < 0.75, "pad": pad,
                "backward": rng.random() < 0.5}
    group = rng.choice([32, 64, 128, 128])
    case = {"op": op, "N": _log_size(rng, 64, 8192), "K": _log_size(rng, 128, 8192, group), "group": group,
            "zero": rng.random() < 0.5, "type": rng.choice(["bf16", "bf16", "fp16"])}
    if op == "quantize":
        return case | {"type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "w4":
        return case | {"M": _log_size(rng, 1, 64), "bias": rng.random() < 0.5}
    while E * case["N"] * case["K"] > 1 << 28:
        E //= 2
    E = max(E, 2)
    return case | {"T": _log_size(rng, 1, 64), "E": E, "k": min(k, E), "bias": rng.random() < 0.5,
                   "gather": rng.random() < 0.5, "pad": pad}


def _pairs(case):
    """Pairs of tokens and experts that are not padding."""
    return (case["T"] - _padding(case)) * case["k"]


def _padding(case):
    return int(case["pad"] * case["T"])


def _experts_used(case):
    """Experts that some pair chooses, about: the others' weights need not be read."""
    E, n = case["E"], _pairs(case)
    return max(min(E, n, case["k"]), int(E * (1 - (1 - 1 / E) ** n)))


def work(case):
    op = case["op"]
    if op == "quantize":
        N, K = case["N"], case["K"]
        # the weight read, codes and scales written, both read again, and the values written
        return {"bytes": N * K * (TYPES[case["type"]].itemsize + 2) + 2 * _w4_bytes(case), "flops": 6 * N * K}
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + _w4_bytes(case) + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        e = TYPES[case["type"]].itemsize
        n = T * E * e + 4 * (E + 1) + 16 * T * k
        if case["backward"]:
            n += T * E * e * (1 if case["normalize"] else 2) + 12 * T * k
        return {"bytes": n, "flops": T * E * (k + 4) * (2 if case["backward"] else 1)}
    R = _pairs(case)
    if op == "combine":
        D, e = case["D"], TYPES[case["type"]].itemsize
        ends = 4 * T * k * (2 if case["weighted"] else 1)
        if case["backward"]:     # dout, and y where its weights have a gradient; dy and dweights
            n = T * D * e + T * k * D * e + ends + (R * D * e + 4 * T * k if case["weighted"] else 0)
            return {"bytes": n, "flops": 3 * R * D}
        return {"bytes": R * D * e + T * D * e + ends, "flops": 2 * R * D}
    N, K, used = case["N"], case["K"], _experts_used(case)
    rows = case["T"] - _padding(case) if case["gather"] else R
    if op == "w4_grouped":
        n = 2 * rows * K + used * _w4_bytes(case) + 2 * T * k * N + (2 * used * N if case["bias"] else 0)
        return {"bytes": n, "flops": 2 * R * N * K}
    if op == "grouped":
        n = 2 * rows * K + 2 * used * N * K + 2 * T * k * N + (2 * used * N if case["bias"] else 0)
        return {"bytes": n, "flops": 2 * R * N * K}
    n = 2 * R * N + 2 * rows * K + 2 * used * N * K + 2 * T * k * K + 2 * E * N * K + (2 * E * N if case["bias"] else 0)
    return {"bytes": n, "flops": 4 * R * N * K}


def _w4_bytes(case):
    """Codes, scales and zero points of one weight."""
    return case["N"] * case["K"] // 2 + case["N"] * case["K"] // case["group"] * (2 + (1 if case["zero"] else 0))


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Hidden states: each token has a magnitude of its own, a few channels are large."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    return x * torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)


def _logits(g, case):
    """A router's logits: some experts are liked more than others; padding tokens choose none."""
    T, E = case["T"], case["E"]
    x = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, E)
    x[T - _padding(case):] = -math.inf
    return x


def prepare(case, seed):
    g = _generator(seed)
    op, s = case["op"], {"case": dict(case)}
    if op == "route":
        s["logits"] = _logits(g, case).to(TYPES[case["type"]])
        if case["backward"]:
            s["dweights"] = 1e-3 * _randn(g, case["T"], case["k"])
        return s
    if op == "quantize":
        s["w"] = (0.02 * _randn(g, case["N"], case["K"]) * torch.exp(0.3 * _randn(g, case["N"], 1))).to(TYPES[case["type"]])
        return s
    t = TYPES[case["type"]]
    if op == "w4":
        s["x"] = _activations(g, case["M"], case["K"]).to(t)
        w = (0.02 * _randn(g, case["N"], case["K"])).to(t)
        s["q"], s["scale"], s["zero"] = _quantize(w, case["group"], case["zero"])
        s["bias"] = _randn(g, case["N"]).to(t) if case["bias"] else None
        return s
    T, E, k = case["T"], case["E"], case["k"]
    _, weights, s["offsets"], s["slots"], rows = _route(_logits(g, case), k, True)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())      # the plain form's capacity of an expert
    if op == "combine":
        s["weights"] = weights if case["weighted"] else None
        s["y"] = _activations(g, T * k, case["D"]).to(t)
        if case["backward"]:
            s["dout"] = (1e-3 * _activations(g, T, case["D"])).to(t)
        return s
    N, K = case["N"], case["K"]
    s["rows"] = rows if case["gather"] else None
    s["A"] = _activations(g, T if case["gather"] else T * k, K).to(t)
    s["bias"] = _randn(g, E, N).to(t) if case["bias"] else None
    if op == "w4_grouped":
        w = (0.02 * _randn(g, E * N, K)).to(t)
        q, scale, zero = _quantize(w, case["group"], case["zero"])
        by_expert = lambda x: x.reshape(-1, E, N).transpose(0, 1).contiguous()       # noqa: E731
        s["q"], s["scale"] = q.reshape(E, N, K // 2), by_expert(scale)
        s["zero"] = None if zero is None else by_expert(zero)
        return s
    s["B"] = (0.02 * _randn(g, E, N, K)).to(t)
    if op == "grouped_backward":
        s["dC"] = (1e-3 * _activations(g, T * k, N)).to(t)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


_ROUTE_OUTPUTS = ("experts", "weights", "offsets", "slots", "rows")


def _own_route(s):
    import persistent_gemm_amd as pg
    c = s["case"]
    got = pg.moe_route(s["logits"], c["k"], normalize=c["normalize"])
    out = dict(zip(_ROUTE_OUTPUTS, got))
    if c["backward"]:
        out["dlogits"] = pg.moe_route_backward(s["dweights"], s["logits"], got[0], got[1], normalize=c["normalize"])
    return out


def _own_grouped(s):
    import persistent_gemm_amd as pg
    return pg.gemm_grouped(s["A"], s["B"], s["offsets"], s["bias"], rows=s["rows"])


def _own_grouped_backward(s):
    import persistent_gemm_amd as pg
    dA, dB, dbias = pg.gemm_grouped_backward(s["dC"], s["A"], s["B"], s["offsets"], rows=s["rows"],
                                             need_dbias=s["case"]["bias"])
    return {"dA": dA, "dB": dB} | ({"dbias": dbias} if s["case"]["bias"] else {})


def _own_combine(s):
    import persistent_gemm_amd as pg
    if not s["case"]["backward"]:
        return pg.moe_combine(s["y"], s["slots"], s["weights"])
    dy, dweights = pg.moe_combine_backward(s["dout"], s["y"], s["slots"], s["weights"], offsets=s["offsets"])
    return {"dy": dy} | ({"dweights": dweights} if s["case"]["weighted"] else {})


def _own_w4(s):
    import persistent_gemm_amd as pg
    return pg.gemm_w4(s["x"], s["q"], s["scale"], s["zero"], s["bias"])


def _own_w4_grouped(s):
    import persistent_gemm_amd as pg
    return pg.gemm_w4(s["A"], s["q"], s["scale"], s["zero"], s["bias"], offsets=s["offsets"], rows=s["rows"])


def _own_quantize(s):
    import persistent_gemm_amd as pg
    c = s["case"]
    q, scale, zero = pg.quantize_w4(s["w"], c["group"], zero=c["zero"])
    out = {"values": pg.dequantize_w4(q, scale, zero), "scale": scale}
    return out | ({"zero": zero} if c["zero"] else {})


# ---------------------------------------------------------------- plain forms

def _route(logits, k, normalize):
    T, E = logits.shape
    x = logits.float()
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    chosen = top > -math.inf
    largest = top[:, :1].clamp(min=torch.finfo(torch.float32).min)
    part = torch.exp(top - largest)
    total = part.sum(dim=1, keepdim=True) if normalize else torch.exp(x - largest).sum(dim=1, keepdim=True)
    weights = torch.where(chosen, part / total, 0.0)
    ids = torch.where(chosen, ids, E)                               # missing choices behind the last expert
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=x.device)
    slots = torch.where(chosen, place.reshape(T, k), -1)
    counts = (flat[:, None] == torch.arange(E, device=x.device)).sum(dim=0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(dim=0)])
    rows = torch.where(flat[order] < E, order // k, -1)
    whole = torch.int32
    return (torch.where(chosen, ids, -1).to(whole), weights, offsets.to(whole), slots.to(whole), rows.to(whole))


def _plain_route(s):
    c, x = s["case"], s["logits"]
    got = _route(x, c["k"], c["normalize"])
    out = dict(zip(_ROUTE_OUTPUTS, got))
    if c["backward"]:
        ids, w, d = got[0].long(), got[1], s["dweights"]
        mean = (w * d).sum(dim=1, keepdim=True)
        # each token's gradients laid out over the experts, with a column more for missing choices
        at = torch.where(ids < 0, c["E"], ids)
        if c["normalize"]:
            full = torch.zeros(c["T"], c["E"] + 1, device=x.device).scatter(1, at, w * (d - mean))[:, :-1]
        else:
            v = x.float()
            p = torch.exp(v - v.amax(dim=1, keepdim=True).clamp(min=torch.finfo(torch.float32).min))
            p = p / p.sum(dim=1, keepdim=True).clamp(min=1e-30)
            full = p * (torch.zeros(c["T"], c["E"] + 1, device=x.device).scatter(1, at, d)[:, :-1] - mean)
        out["dlogits"] = full.to(x.dtype)
    return out


def _places(s):
    """(expert, place within it) of each row; rows behind the last expert's go to an expert of their own."""
    o = s["offsets"].long()
    R, E = s["case"]["T"] * s["case"]["k"], s["case"]["E"]
    r = torch.arange(R, device=o.device)
    e = (r[:, None] >= o[1:]).sum(dim=1)
    start = torch.cat([o, o[-1:]])[e]
    return e, torch.where(e < E, r - start, 0)


def _padded(x, e, at, s):
    """Rows by expert, [E, most, columns], zeros where an expert has fewer."""
    out = torch.zeros(s["case"]["E"] + 1, s["most"], x.shape[1], device=x.device)
    out[e, at] = x.float()
    return out[:-1]


def _rows_of(s):
    return s["A"] if s["rows"] is None else s["A"][s["rows"].long().clamp(min=0)]


def _from_experts(c, e, at):
    """Padded rows back in their order, zeros behind the last expert's."""
    last = e.clamp(max=c.shape[0] - 1)
    return torch.where((e < c.shape[0])[:, None], c[last, at], 0.0)


def _product(s, b):
    e, at = _places(s)
    c = torch.bmm(_padded(_rows_of(s), e, at, s), b.transpose(1, 2))
    if s["bias"] is not None:
        c = c + s["bias"].float()[:, None]
    return _from_experts(c, e, at).to(s["A"].dtype)


def _plain_grouped(s):
    return _product(s, s["B"].float())


def _plain_grouped_backward(s):
    e, at = _places(s)
    d, a = _padded(s["dC"], e, at, s), _padded(_rows_of(s), e, at, s)
    t = s["A"].dtype
    out = {"dA": _from_experts(torch.bmm(d, s["B"].float()), e, at).to(t), "dB": torch.bmm(d.transpose(1, 2), a).to(t)}
    return out | ({"dbias": d.sum(dim=1).to(t)} if s["case"]["bias"] else {})


def _plain_combine(s):
    slots = s["slots"].long()
    there = (slots >= 0)[:, :, None]
    w = 1.0 if s["weights"] is None else s["weights"][:, :, None]
    y = s["y"]
    if not s["case"]["backward"]:
        return torch.where(there, y[slots.clamp(min=0)].float() * w, 0.0).sum(dim=1).to(y.dtype)
    d = s["dout"].float()[:, None]
    at = torch.where(slots < 0, y.shape[0], slots)              # a row more for missing choices
    dy = torch.zeros(y.shape[0] + 1, y.shape[1], device=y.device)
    dy[at] = d * w
    out = {"dy": dy[:-1].to(y.dtype)}
    if s["case"]["weighted"]:
        out["dweights"] = torch.where(there, y[slots.clamp(min=0)].float() * d, 0.0).sum(dim=2)
    return out


def _scale_type(w):
    return torch.bfloat16 if w.dtype == torch.float32 else w.dtype


def _quantize(w, group, zero):
    """Codes [N, K / 2] (the even element in the low half of a byte), 16-bit scales [K / group, N], zero points."""
    N, K = w.shape
    g = w.float().reshape(N, K // group, group)
    t = _scale_type(w)
    smallest = torch.finfo(t).tiny
    if zero:       # codes 0 .. 15 over [min(0, smallest), max(0, largest)]
        lo, hi = g.amin(dim=2).clamp(max=0.0), g.amax(dim=2).clamp(min=0.0)
        scale = ((hi - lo) / 15.0).to(t).clamp(min=smallest)
        z = torch.round(-lo.double() / scale.double()).clamp(0, 15)
    else:          # codes 1 .. 15 with 8 for zero
        scale = (g.abs().amax(dim=2) / 7.0).to(t).clamp(min=smallest)
        z = torch.full_like(scale, 8.0, dtype=torch.float64)
    # the quotient in 64 bits: it may lie on the border between two codes, or next to it
    q = (torch.round(g.double() / scale.double()[:, :, None]) + z[:, :, None]).clamp(0, 15)
    q = q.to(torch.uint8).reshape(N, K // 2, 2)
    return (q[:, :, 0] | q[:, :, 1] << 4, scale.t().contiguous(), z.to(torch.uint8).t().contiguous() if zero else None)


def _values(q, scale, zero):
    """fp32 values of codes [..., N, K / 2] with scales [..., groups, N]."""
    v = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2).float()
    v = v.unflatten(-1, (scale.shape[-2], -1))
    z = 8.0 if zero is None else zero.float().transpose(-1, -2)[..., None]
    return ((v - z) * scale.float().transpose(-1, -2)[..., None]).flatten(-2)


def _plain_w4(s):
    c = s["x"].float() @ _values(s["q"], s["scale"], s["zero"]).t()
    if s["bias"] is not None:
        c = c + s["bias"].float()
    return c.to(s["x"].dtype)


def _plain_w4_grouped(s):
    return _product(s, _values(s["q"], s["scale"], s["zero"]))


def _plain_quantize(s):
    q, scale, zero = _quantize(s["w"], s["case"]["group"], s["case"]["zero"])
    out = {"values": _values(q, scale, zero).to(scale.dtype), "scale": scale}
    return out | ({"zero": zero} if s["case"]["zero"] else {})


_OWN = {"route": _own_route, "grouped": _own_grouped, "grouped_backward": _own_grouped_backward, "combine": _own_combine,
        "w4": _own_w4, "w4_grouped": _own_w4_grouped, "quantize": _own_quantize}
_PLAIN = {"route": _plain_route, "grouped": _plain_grouped, "grouped_backward": _plain_grouped_backward,
          "combine": _plain_combine, "w4": _plain_w4, "w4_grouped": _plain_w4_grouped, "quantize": _plain_quantize}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_route(s):
    """The choices one after the other, each the first of the largest logits that are left."""
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].double()
    left, ids = x.clone(), []
    index = torch.arange(E, device=x.device)
    for _ in range(k):
        best = left.amax(dim=1, keepdim=True)
        first = torch.where(left == best, index, E).amin(dim=1)
        ids.append(torch.where(best[:, 0] == -math.inf, -1, first))
        left[torch.arange(T, device=x.device), first] = -math.inf
    ids = torch.stack(ids, dim=1)
    chosen = torch.zeros(T, E, dtype=torch.bool, device=x.device)
    for j in range(k):
        chosen |= ids[:, j:j + 1] == index
    e = torch.exp(x - x.amax(dim=1, keepdim=True)).nan_to_num(0.0)       # a token without choices: all 0
    total = (e * chosen if c["normalize"] else e).sum(dim=1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    w = torch.where(ids < 0, 0.0, p.gather(1, ids.clamp(min=0)))
    slots, rows = torch.full_like(ids, -1), torch.full((T * k,), -1, device=x.device)
    offsets = [0]
    for n in range(E):
        t, j = torch.nonzero(ids == n, as_tuple=True)
        at = offsets[-1] + torch.arange(t.numel(), device=x.device)
        slots[t, j] = at
        rows[at] = t
        offsets.append(offsets[-1] + t.numel())
    whole = torch.int32
    out = {"experts": ids.to(whole), "weights": w, "offsets": torch.tensor(offsets, dtype=whole, device=x.device),
           "slots": slots.to(whole), "rows": rows.to(whole)}
    if c["backward"]:
        d = torch.zeros(T, E, dtype=torch.float64, device=x.device)
        for j in range(k):
            d += torch.where(ids[:, j:j + 1] == index, s["dweights"][:, j:j + 1].double(), 0.0)
        kept = p * chosen if c["normalize"] else p
        out["dlogits"] = kept * (d - (p * chosen * d).sum(dim=1, keepdim=True))
    return out


def _groups(s):
    """(expert, first row, end) of each expert with rows."""
    o = s["offsets"].tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e] < o[e + 1]]


def _tokens_64(s, a, b):
    return (s["A"][a:b] if s["rows"] is None else s["A"][s["rows"][a:b].long()]).double()


def _exact_product(s, weight_of):
    R, N = s["case"]["T"] * s["case"]["k"], s["case"]["N"]
    c = torch.zeros(R, N, dtype=torch.float64, device=s["A"].device)
    for e, a, b in _groups(s):
        c[a:b] = torch.mm(_tokens_64(s, a, b), weight_of(e).t())
        if s["bias"] is not None:
            c[a:b] += s["bias"][e].double()
    return c


def _exact_grouped(s):
    return _exact_product(s, lambda e: s["B"][e].double())


def _exact_grouped_backward(s):
    c, dev = s["case"], s["A"].device
    dA = torch.zeros(c["T"] * c["k"], c["K"], dtype=torch.float64, device=dev)
    dB = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device=dev)
    dbias = torch.zeros(c["E"], c["N"], dtype=torch.float64, device=dev)
    for e, a, b in _groups(s):
        d = s["dC"][a:b].double()
        dA[a:b] = torch.mm(d, s["B"][e].double())
        dB[e] = torch.mm(d.t().contiguous(), _tokens_64(s, a, b))
        dbias[e] = d.sum(dim=0)
    return {"dA": dA, "dB": dB} | ({"dbias": dbias} if c["bias"] else {})


def _exact_combine(s):
    c = s["case"]
    slots, y = s["slots"].long(), s["y"].double()
    w = torch.ones_like(slots, dtype=torch.float64) if s["weights"] is None else s["weights"].double()
    out = torch.zeros(c["T"], c["D"], dtype=torch.float64, device=y.device)
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(c["k"]):
        t = torch.nonzero(slots[:, j] >= 0)[:, 0]
        at = slots[t, j]
        if c["backward"]:
            d = s["dout"][t].double()
            dy[at] = w[t, j, None] * d
            dw[t, j] = torch.linalg.vecdot(d, y[at])
        else:
            out[t] += w[t, j, None] * y[at]
    if not c["backward"]:
        return out
    return {"dy": dy} | ({"dweights": dw} if c["weighted"] else {})


def _weight_64(q, scale, zero, group):
    """One weight's values from its codes."""
    v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = (q % 16).double(), torch.div(q, 16, rounding_mode="floor").double()
    v -= 8.0 if zero is None else zero.double().repeat_interleave(group, dim=0).t()
    return v * scale.double().repeat_interleave(group, dim=0).t()


def _exact_w4(s):
    c = torch.mm(s["x"].double(), _weight_64(s["q"], s["scale"], s["zero"], s["case"]["group"]).t())
    return c if s["bias"] is None else c + s["bias"].double()


def _exact_w4_grouped(s):
    zero = lambda e: None if s["zero"] is None else s["zero"][e]       # noqa: E731
    return _exact_product(s, lambda e: _weight_64(s["q"][e], s["scale"][e], zero(e), s["case"]["group"]))


def _exact_quantize(s):
    c, w = s["case"], s["w"].double()
    K, group, t = c["K"], c["group"], _scale_type(s["w"])
    scales, zeros, values = [], [], []
    for k in range(0, K, group):
        part = w[:, k:k + group]
        if c["zero"]:
            top, low = part.amax(dim=1).clamp(min=0), part.amin(dim=1).clamp(max=0)
            unit, codes = top - low, 15
        else:
            unit, codes = part.abs().amax(dim=1), 7
        scale = (unit / codes).float().to(t).double().clamp(min=torch.finfo(t).tiny)
        z = torch.round(-low / scale).clamp(0, 15) if c["zero"] else torch.full_like(scale, 8.0)
        code = (torch.round(part / scale[:, None]) + z[:, None]).clamp(0, 15)
        scales.append(scale)
        zeros.append(z)
        values.append((code - z[:, None]) * scale[:, None])
    out = {"values": torch.cat(values, dim=1), "scale": torch.stack(scales)}
    return out | ({"zero": torch.stack(zeros).to(torch.uint8)} if c["zero"] else {})


_EXACT = {"route": _exact_route, "grouped": _exact_grouped, "grouped_backward": _exact_grouped_backward,
          "combine": _exact_combine, "w4": _exact_w4, "w4_grouped": _exact_w4_grouped, "quantize": _exact_quantize}
