"""Timed cases of the block-scaled fp8 operators and the norms around a block.

The operators, with s the fp32 scale of a block of 128 (rows of the operand by 128 along K, or
128 x 128), q E4M3 codes, and everything summed in 32 bits or more:

- ``quantize_fp8_block``: s = max(max|x| / 448, 2^-126) over the block, q the E4M3 value nearest to x / s;
- ``gemm_fp8_block``: C[m, n] = sum_b sA[b, m] sB[., b] sum_{k in b} qA[m, k] qB[n, k] + bias[n];
- ``gemm_fp8_block_backward``: dA = q(dC) . B, dB = q(dC)^T . A, dbias = column sums of dC, where q()
  quantises dC along the dimension that the product sums over;
- ``rms_norm`` (before a block): y = x rstd w, rstd = (mean x^2 + eps)^-1/2, as it is or quantised in
  blocks of 128 for the product that follows;
- ``gated_norm`` (after a block): out = residual_scale * residual + gate * (h rstd w), optionally with
  the next block's ``rms_norm`` of the stored out in the same pass; both with their gradients.
"""

import math

import torch

own = False

EPS = 1e-6
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -126
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a small projection: latency of one call
        {"name": "gemm 256x256x512", "op": "gemm", "M": 256, "N": 256, "K": 512, "bias": True, "b": "tile"},
        # one token through a square projection: the weights are read once
        {"name": "gemm 1x4096x4096", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "bias": False, "b": "tile"},
        # a decode batch through a wide projection
        {"name": "gemm 16x8192x8192", "op": "gemm", "M": 16, "N": 8192, "K": 8192, "bias": False, "b": "tile"},
        # a ragged prefill: no size is a multiple of a tile, K ends inside a block
        {"name": "gemm 777x4099x2060", "op": "gemm", "M": 777, "N": 4099, "K": 2060, "bias": True, "b": "tile"},
        # a full prefill or training batch
        {"name": "gemm 8192x8192x8192", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "bias": True, "b": "tile"},
        # the backward of a training step's projection
        {"name": "gemm backward 4096x4096x4096", "op": "gemm_backward", "M": 4096, "N": 4096, "K": 4096},
        # the same for a ragged batch of tokens and odd widths
        {"name": "gemm backward 1037x2050x1290", "op": "gemm_backward", "M": 1037, "N": 2050, "K": 1290},
        # activations for the forward product and, transposed, for the weight gradient
        {"name": "quantize 8192x8192 both", "op": "quantize", "R": 8192, "C": 8192, "block": "row",
         "transpose": "both", "type": "bf16"},
        # a weight of odd sizes after an optimizer step in fp32
        {"name": "quantize tile 1000x2051", "op": "quantize", "R": 1000, "C": 2051, "block": "tile",
         "transpose": "both", "type": "fp32"},
        # decode: the norm before a block, straight to fp8
        {"name": "norm fp8 16x8192", "op": "norm", "T": 16, "D": 8192, "gate": "none", "post": False, "pre": True,
         "fp8": True, "scaled": False, "type": "bf16"},
        # training, forward: the norm after a block, gated per sequence, and the next block's norm to fp8
        {"name": "gated norm fp8 16384x4096", "op": "norm", "T": 16384, "D": 4096, "gate": "sequence", "post": True,
         "pre": True, "fp8": True, "scaled": True, "type": "bf16"},
        # training, backward of both norms at odd sizes in fp32
        {"name": "norm backward 4095x2047", "op": "norm_backward", "T": 4095, "D": 2047, "gate": "vector",
         "post": True, "pre": True, "scaled": True, "type": "fp32"},
    ]


def _log_size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    if rng.random() < 0.5 and n >= 256:      # half of the larger ones are the usual multiples
        n -= n % 128
    return n + 128 if n == 24 * 128 else n


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm_backward", "quantize", "norm", "norm_backward"])
    if op == "gemm":
        return {"op": op, "M": _log_size(rng, 1, 8192), "N": _log_size(rng, 64, 8192), "K": _log_size(rng, 64, 8192),
                "bias": rng.random() < 0.5, "b": rng.choice(["tile", "tile", "row"])}
    if op == "gemm_backward":
        return {"op": op, "M": _log_size(rng, 16, 4096), "N": _log_size(rng, 64, 4096), "K": _log_size(rng, 64, 4096)}
    if op == "quantize":
        return {"op": op, "R": _log_size(rng, 1, 8192), "C": _log_size(rng, 64, 8192),
                "block": rng.choice(["row", "tile"]), "transpose": rng.choice(["no", "yes", "both"]),
                "type": rng.choice(["bf16", "bf16", "fp32"])}
    post = rng.random() < 0.7
    pre = not post or rng.random() < 0.5
    case = {"op": op, "T": _log_size(rng, 1, 8192), "D": _log_size(rng, 64, 8192),
            "gate": rng.choice(["none", "vector", "token"]) if post else "none", "post": post, "pre": pre,
            "scaled": post and rng.random() < 0.5, "type": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "norm":
        case["fp8"] = pre and rng.random() < 0.5
    return case


def _up(n, m):
    return -(-n // m) * m


def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], _up(case["K"], 16)
        kb = _up(K, 128) // 128
        scales = 4 * kb * (M + (N if case["b"] == "row" else _up(N, 128) // 128))
        return {"bytes": (M + N) * K + scales + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "gemm_backward":
        M, N, K = case["M"], case["N"], case["K"]
        mb, nb, kb = (_up(n, 128) // 128 for n in (M, N, K))
        read = 2 * M * N + K * _up(M, 16) + K * _up(N, 16) + 4 * (mb * K + nb * kb)
        return {"bytes": read + 2 * (M * K + N * K + N), "flops": 4 * M * N * K}
    if op == "quantize":
        R, C = case["R"], case["C"]
        rb, cb = _up(R, 128) // 128, _up(C, 128) // 128
        n = R * C * TYPES[case["type"]].itemsize
        if case["transpose"] in ("no", "both"):
            n += R * _up(C, 16) + 4 * cb * (R if case["block"] == "row" else rb)
        if case["transpose"] in ("yes", "both"):
            n += C * _up(R, 16) + 4 * rb * (C if case["block"] == "row" else cb)
        return {"bytes": n, "flops": 4 * R * C}
    T, D, e = case["T"], case["D"], TYPES[case["type"]].itemsize
    rows = {"none": 0, "vector": 1, "sequence": case.get("G", _sequences(T)), "token": T}[case["gate"]]
    both = case["post"] and case["pre"]
    vectors = int(case["post"]) + int(case["pre"]) + int(case["scaled"])
    if op == "norm":
        n = T * D * e * (2 if case["post"] else 1) + (vectors + rows) * D * e       # h and residual, or x
        n += T * D * e * int(case["post"]) + 4 * T * (1 + int(both))               # out, rstd
        if case["pre"]:
            n += T * _up(D, 16) + 4 * T * (_up(D, 128) // 128) if case["fp8"] else T * D * e
        return {"bytes": n, "flops": T * D * (8 * int(case["post"]) + 5 * int(case["pre"]))}
    # gradients: dy and x (or out), dout, h, and residual where its scale has a gradient; written: dx or dh and dresidual
    n = T * D * e * (2 * int(case["pre"]) + 1 + int(case["post"]) + int(case["scaled"]))
    n += T * D * e * (2 if case["post"] else 1) + 2 * (vectors + rows) * D * e + 4 * T * (1 + int(both))
    return {"bytes": n, "flops": T * D * (14 * int(case["post"]) + 9 * int(case["pre"]))}


def _sequences(T):
    """Sequences of a batch of T tokens that share one gate each."""
    return 8 if T % 8 == 0 else 1


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Hidden states: each token has a magnitude of its own, a few channels are large."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    return x * torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)


def prepare(case, seed):
    g = _generator(seed)
    op, state = case["op"], {"case": dict(case)}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        state["A"], state["A_scale"] = _quantize_rows(_activations(g, M, K))
        w = _randn(g, N, K) * 0.02
        state["B"], state["B_scale"] = _quantize_rows(w) if case["b"] == "row" else _quantize_tiles(w)
        state["bias"] = _randn(g, N).to(torch.bfloat16) if case["bias"] else None
    elif op == "gemm_backward":
        M, N, K = case["M"], case["N"], case["K"]
        state["dC"] = (_activations(g, M, N) * 1e-3).to(torch.bfloat16)
        state["At"], state["At_scale"] = _quantize_rows(_activations(g, M, K).t())
        state["Bt"], state["Bt_scale"] = _quantize_tiles((_randn(g, N, K) * 0.02).t())
    elif op == "quantize":
        x = _activations(g, case["R"], case["C"])
        state["x"] = (x if case["block"] == "row" else x * 0.02).to(TYPES[case["type"]])
    else:
        T, D, t = case["T"], case["D"], TYPES[case["type"]]
        G = {"none": 0, "vector": 1, "sequence": _sequences(T), "token": T}[case["gate"]]
        state["weight"] = (1 + 0.1 * _randn(g, D)).to(t)
        state["next_weight"] = (1 + 0.1 * _randn(g, D)).to(t)
        state["gate"] = (0.5 + 0.2 * _randn(g, G, D)).to(t) if G else None
        state["residual_scale"] = (1 + 0.05 * _randn(g, D)).to(t) if case["scaled"] else None
        state["residual"] = (3 * _activations(g, T, D)).to(t)
        state["h"] = _activations(g, T, D).to(t) if case["post"] else None
        if op == "norm_backward":
            fwd = _plain_norm(dict(state, case=dict(case, fp8=False)))
            state["out"] = fwd["out"] if case["post"] else state["residual"]
            state["rstd"], state["rstd_next"] = fwd.get("rstd"), fwd.get("rstd_next")
            state["dout"] = (1e-3 * _activations(g, T, D)).to(t)
            state["dy"] = (1e-3 * _activations(g, T, D)).to(t) if case["pre"] else None
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_gemm(s):
    import persistent_gemm_amd as pg
    return pg.gemm_fp8_block(s["A"], s["B"], s["A_scale"], s["B_scale"], s["bias"])


def _own_gemm_backward(s):
    import persistent_gemm_amd as pg
    dA, dB, dbias = pg.gemm_fp8_block_backward(s["dC"], s["At"], s["At_scale"], s["Bt"], s["Bt_scale"])
    return {"dA": dA, "dB": dB, "dbias": dbias}


def _own_quantize(s):
    import persistent_gemm_amd as pg
    c = s["case"]
    return pg.quantize_fp8_block(s["x"], c["block"], transpose={"no": False, "yes": True, "both": "both"}[c["transpose"]])


def _own_norm(s):
    import persistent_gemm_amd as pg
    c = s["case"]
    if not c["post"]:
        got = pg.rms_norm(s["residual"], s["next_weight"], EPS, quantize=c["fp8"])
        return dict(zip(("q", "scale", "rstd_next") if c["fp8"] else ("y", "rstd_next"), got))
    got = pg.gated_norm(s["h"], s["residual"], s["weight"], s["gate"], s["residual_scale"], EPS,
                        next_weight=s["next_weight"] if c["pre"] else None, quantize=c["pre"] and c["fp8"])
    names = ("out", "rstd")
    if c["pre"]:
        names += ("q", "scale", "rstd_next") if c["fp8"] else ("y", "rstd_next")
    return dict(zip(names, got))


def _own_norm_backward(s):
    import persistent_gemm_amd as pg
    c = s["case"]
    if not c["post"]:
        dx, dw = pg.rms_norm_backward(s["dy"], s["out"], s["next_weight"], s["rstd_next"], dresidual=s["dout"])
        return {"dx": dx, "dnext_weight": dw}
    nxt = {"dy": s["dy"], "out": s["out"], "next_weight": s["next_weight"], "rstd_next": s["rstd_next"]} if c["pre"] else {}
    got = pg.gated_norm_backward(s["dout"], s["h"], s["weight"], s["rstd"], s["gate"], s["residual"],
                                 s["residual_scale"], **nxt)
    names = ("dh", "dresidual", "dweight", "dgate", "dresidual_scale", "dnext_weight")
    return {n: v for n, v in zip(names, got) if v is not None}


# ---------------------------------------------------------------- plain forms

def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _scale_of(amax):
    s = (amax.double() / 448.0).float().clamp(min=TINY)     # the quotient, rounded once
    return torch.where(torch.isfinite(s), s, math.nan)


def _codes(x, s):
    """E4M3 codes nearest to x / s, ties to even.  The quotient is held in 64 bits: x / s lies on or
    next to the border between two codes for many x (448 x / max|x| is a short binary fraction)."""
    v = x.double() / s.double()
    exponent = torch.frexp(v).exponent.clamp(min=-5) - 4        # of a code's last place
    step = ((exponent.long() + 1023) << 52).view(torch.float64)  # 2^exponent
    return (torch.round(v / step) * step).to(E4M3)


def _quantize_rows(x):
    """[R, C] -> codes [R, C up to 16], scales [blocks, R]: blocks of 128 along a row."""
    R, C = x.shape
    x = _pad(x.float(), R, _up(C, 128)).reshape(R, -1, 128)
    s = _scale_of(x.abs().amax(dim=2, keepdim=True))
    q = _codes(x, s).reshape(R, -1)[:, :_up(C, 16)].contiguous()
    return q, s[:, :, 0].t().contiguous()


def _quantize_tiles(x):
    """[R, C] -> codes [R, C up to 16], scales [row blocks, column blocks]."""
    R, C = x.shape
    x = _pad(x.float(), _up(R, 128), _up(C, 128)).reshape(_up(R, 128) // 128, 128, -1, 128)
    s = _scale_of(x.abs().amax(dim=(1, 3), keepdim=True))
    q = _codes(x, s).reshape(_up(R, 128), -1)[:R, :_up(C, 16)].contiguous()
    return q, s[:, 0, :, 0].contiguous()


def _dequantize(q, scale, by_row):
    """fp32 values of codes [R, Kp] with scales [blocks, R] (by_row) or [row blocks, blocks]."""
    R, K = q.shape
    if by_row:
        s = scale.t().repeat_interleave(128, dim=1)[:, :K]
    else:
        s = scale.repeat_interleave(128, dim=0)[:R].repeat_interleave(128, dim=1)[:, :K]
    return q.float() * s


def _plain_gemm(s):
    a = _dequantize(s["A"], s["A_scale"], True)
    b = _dequantize(s["B"], s["B_scale"], s["case"]["b"] == "row")
    c = a @ b.t()
    if s["bias"] is not None:
        c = c + s["bias"].float()
    return c.to(torch.bfloat16)


def _plain_gemm_backward(s):
    dc = s["dC"]
    M, N = dc.shape
    along_n = _dequantize(*_quantize_rows(dc), True)[:, :N]
    along_m = _dequantize(*_quantize_rows(dc.t()), True)[:, :M]
    at = _dequantize(s["At"], s["At_scale"], True)[:, :M]
    bt = _dequantize(s["Bt"], s["Bt_scale"], False)[:, :N]
    out = {"dA": along_n @ bt.t(), "dB": along_m @ at.t(), "dbias": dc.float().sum(dim=0)}
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


def _plain_quantize(s):
    c, x = s["case"], s["x"]
    form = _quantize_rows if c["block"] == "row" else _quantize_tiles
    out = ()
    if c["transpose"] != "yes":
        out += form(x)
    if c["transpose"] != "no":
        out += form(x.t())
    return out


def _gate_rows(gate, T):
    """The gate of each token, [T, D] or [1, D]: row t // (T / G)."""
    g = gate.float()
    return g if g.shape[0] in (1, T) else g.repeat_interleave(T // g.shape[0], dim=0)


def _plain_norm(s):
    c, t, out = s["case"], s["residual"].dtype, {}
    x = s["residual"]
    if c["post"]:
        h = s["h"].float()
        r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        n = h * r * s["weight"].float()
        if s["gate"] is not None:
            n = n * _gate_rows(s["gate"], h.shape[0])
        res = x.float()
        if s["residual_scale"] is not None:
            res = res * s["residual_scale"].float()
        x = (res + n).to(t)
        out["out"], out["rstd"] = x, r[:, 0]
    if c["pre"]:
        v = x.float()
        r = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        y = v * r * s["next_weight"].float()
        if c["fp8"]:
            out["q"], out["scale"] = _quantize_rows(y)
        else:
            out["y"] = y.to(t)
        out["rstd_next"] = r[:, 0]
    return out


def _plain_norm_backward(s):
    c, t, out = s["case"], s["residual"].dtype, {}
    dv = s["dout"].float()
    if c["pre"]:
        dy, xh = s["dy"].float(), s["out"].float() * s["rstd_next"][:, None]
        out["dnext_weight"] = (dy * xh).sum(dim=0)
        gr = dy * s["next_weight"].float()
        dv = dv + s["rstd_next"][:, None] * (gr - xh * (gr * xh).mean(dim=1, keepdim=True))
    if not c["post"]:
        out["dx"] = dv
        return {k: v.to(t) for k, v in out.items()}
    T, D = dv.shape
    hh, w = s["h"].float() * s["rstd"][:, None], s["weight"].float()
    dn = dv
    if s["gate"] is not None:
        dn = dv * _gate_rows(s["gate"], T)
        out["dgate"] = (dv * hh * w).reshape(s["gate"].shape[0], -1, D).sum(dim=1)
    out["dweight"] = (dn * hh).sum(dim=0)
    gr = dn * w
    out["dh"] = s["rstd"][:, None] * (gr - hh * (gr * hh).mean(dim=1, keepdim=True))
    out["dresidual"] = dv
    if s["residual_scale"] is not None:
        out["dresidual_scale"] = (dv * s["residual"].float()).sum(dim=0)
        out["dresidual"] = dv * s["residual_scale"].float()
    return {k: v.to(t) for k, v in out.items()}


_OWN = {"gemm": _own_gemm, "gemm_backward": _own_gemm_backward, "quantize": _own_quantize, "norm": _own_norm,
        "norm_backward": _own_norm_backward}
_PLAIN = {"gemm": _plain_gemm, "gemm_backward": _plain_gemm_backward, "quantize": _plain_quantize,
          "norm": _plain_norm, "norm_backward": _plain_norm_backward}


# ---------------------------------------------------------------- in 64 bits

def _e4m3_64(v):
    """v rounded to the nearest E4M3 value, ties to the even code, from the table of all its magnitudes."""
    table = torch.arange(127, dtype=torch.uint8, device=v.device).view(E4M3).double()
    borders = (table[1:] + table[:-1]) / 2
    a = v.abs().contiguous()
    below = torch.bucketize(a, borders)                          # borders under a
    tie = torch.bucketize(a, borders, right=True) - below        # 1 where a is a border
    return torch.copysign(table[below + tie * (below % 2)], v)


def _blocks_64(x, rows):
    """(values of the codes, unrounded scale of each block), both at x's size, blocks of rows x 128."""
    R, C = x.shape
    q, s = torch.zeros(R, _up(C, 16), dtype=torch.float64, device=x.device), []
    for c0 in range(0, C, 128):
        part = x[:, c0:c0 + 128].double()
        a = part.abs().amax(dim=1)
        if rows > 1:
            a = _pad(a[:, None], _up(R, rows), 1).reshape(-1, rows).amax(dim=1)
        s.append((a / 448.0).clamp(min=TINY))
        stored = s[-1].float().double()      # what is kept is the scale in fp32
        q[:, c0:c0 + part.shape[1]] = _e4m3_64(part / stored.repeat_interleave(rows)[:R, None])
    return q, torch.stack(s)                 # scales [column blocks, rows or row blocks]


def _values_64(q, scale_by_block):
    """Values of codes [R, Kp] from fp32 scales [column blocks, R or row blocks], as kept."""
    v, R = q.double(), q.shape[0]
    for b in range(scale_by_block.shape[0]):
        s = scale_by_block[b].float().double()
        if s.shape[0] != R:
            s = s.repeat_interleave(128)[:R]
        v[:, 128 * b:128 * b + 128] *= s[:, None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        b_scale = s["B_scale"] if case["b"] == "row" else s["B_scale"].t()
        c = torch.mm(_values_64(s["A"], s["A_scale"]), _values_64(s["B"], b_scale).t())
        return c if s["bias"] is None else c + s["bias"].double()
    if op == "gemm_backward":
        dc = s["dC"]
        M, N = dc.shape
        dn = _values_64(*_blocks_64(dc, 1))[:, :N]
        dm = _values_64(*_blocks_64(dc.t(), 1))[:, :M]
        at = _values_64(s["At"], s["At_scale"])[:, :M]
        bt = _values_64(s["Bt"], s["Bt_scale"].t())[:, :N]
        return {"dA": torch.mm(dn, bt.t()), "dB": torch.mm(dm, at.t()), "dbias": dc.double().sum(dim=0)}
    if op == "quantize":
        out, rows = (), 1 if case["block"] == "row" else 128
        for x in {"no": (s["x"],), "yes": (s["x"].t(),), "both": (s["x"], s["x"].t())}[case["transpose"]]:
            q, scale = _blocks_64(x, rows)
            out += (q, scale if rows == 1 else scale.t().contiguous())
        return out
    return _exact_norm(s) if op == "norm" else _exact_norm_backward(s)


def _unit_64(x):
    """(x / its root mean square, 1 / that root), eps inside."""
    x = x.double()
    r = 1.0 / torch.sqrt(x.square().sum(dim=1) / x.shape[1] + EPS)
    return x * r[:, None], r


def _token_gate_64(s, T):
    if s["gate"] is None:
        return torch.ones(1, 1, dtype=torch.float64, device=s["residual"].device)
    rows = torch.arange(T, device=s["gate"].device) * s["gate"].shape[0] // T
    return s["gate"].double()[rows]


def _exact_norm(s):
    c, x, out = s["case"], s["residual"], {}
    if c["post"]:
        unit, out["rstd"] = _unit_64(s["h"])
        keep = 1.0 if s["residual_scale"] is None else s["residual_scale"].double()
        out["out"] = keep * x.double() + _token_gate_64(s, x.shape[0]) * (s["weight"].double() * unit)
        x = out["out"].to(x.dtype)           # the next norm reads what is stored
    if c["pre"]:
        unit, out["rstd_next"] = _unit_64(x)
        y = unit * s["next_weight"].double()
        if c["fp8"]:
            out["q"], out["scale"] = _blocks_64(y, 1)
        else:
            out["y"] = y
    return out


def _through_norm_64(grad, unit, r):
    """The gradient at a norm's input from `grad` at its unit output."""
    return r[:, None] * (grad - unit * ((grad * unit).sum(dim=1, keepdim=True) / unit.shape[1]))


def _exact_norm_backward(s):
    c, out = s["case"], {}
    d = s["dout"].double()
    if c["pre"]:
        r = s["rstd_next"].double()
        unit, dy = s["out"].double() * r[:, None], s["dy"].double()
        out["dnext_weight"] = (unit * dy).sum(dim=0)
        d = _through_norm_64(s["next_weight"].double() * dy, unit, r) + d
    if not c["post"]:
        out["dx"] = d
        return out
    r, w = s["rstd"].double(), s["weight"].double()
    unit, gate = s["h"].double() * r[:, None], _token_gate_64(s, d.shape[0])
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        out["dgate"] = (d * unit).reshape(G, -1, d.shape[1]).sum(dim=1) * w
    out["dweight"] = (d * gate * unit).sum(dim=0)
    out["dh"] = _through_norm_64(d * gate * w, unit, r)
    out["dresidual"] = d
    if s["residual_scale"] is not None:
        out["dresidual_scale"] = (s["residual"].double() * d).sum(dim=0)
        out["dresidual"] = s["residual_scale"].double() * d
    return out
