"""A layer of experts: routing, products grouped by expert, and products with 4-bit weights.

Every call runs in the library's HIP kernels (``include/sk_gemm.h`` has layouts and limits) and uses no scratch of the
library, so all of them may be captured into a HIP graph.  Outputs are allocated on the stream that the call uses.  Tensors
are contiguous, and every size is at least 1: a call without rows or tokens raises.
"""

from __future__ import annotations

import contextlib

import persistent_gemm_amd as _pg

__all__ = ["moe_route", "moe_route_backward", "moe_combine", "moe_combine_backward", "gemm_grouped",
           "gemm_grouped_backward", "gemm_w4", "quantize_w4", "dequantize_w4"]

_HERE = contextlib.nullcontext()


def _on(t, name, stream):
    """A context in which t's device is the current one and `stream` (a torch stream, a handle, or None: the device's
    current stream) the current stream: outputs are allocated and kernels launched there."""
    torch = _pg._torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}, expected a GPU")
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_pg._handle(stream), device=t.device)
        elif stream.device != t.device:
            raise ValueError(f"stream is of {stream.device}, {name} on {t.device}")
        return torch.cuda.stream(stream)
    return _HERE if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def _integer(v, name):
    n = int(v)
    if n != v:
        raise ValueError(f"{name} is {v!r}, expected a whole number")
    return n


def _types(t, name, full=True):
    """SK_ELEM_* of a tensor."""
    torch = _pg._torch()
    elems = {torch.bfloat16: 0, torch.float16: 2, torch.float32: 1}
    if not full:
        del elems[torch.float32]
    if t.dtype not in elems:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(elems)}")
    return elems[t.dtype]


def _dims(t, name, n):
    if not isinstance(t, _pg._torch().Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() not in (n if isinstance(n, tuple) else (n,)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {n} dimensions")
    return t.shape


def _whole(t, name, shape, dev):
    _pg._need(t, name, (_pg._torch().int32,), shape, dev)


def _optional(t, name, types, shape, dev):
    if t is not None:
        _pg._need(t, name, types, shape, dev)


def _run(name, *args):
    _pg._ok(getattr(_pg.load(), name)(*args), name)


# ---------------------------------------------------------------- routing

def moe_route(logits, k, *, normalize=True, stream=None):
    """The k largest of each token's logits [T, E] (bf16, fp16 or fp32) and the order of the pairs (token, choice) by
    expert: (experts, weights, offsets, slots, rows).

    experts int32 [T, k]: the choices in falling order, ties to the lower expert; an expert whose logit is -inf or NaN is
    never chosen, and where none is left the choice is -1.  weights fp32 [T, k]: their softmax over the chosen ones
    (normalize=True) or over all E; 0 without an expert, NaN for a token with a NaN logit.  offsets int32 [E + 1],
    slots int32 [T, k], rows int32 [T * k]: pair (t, j) is row slots[t, j] (-1 without an expert) of the rows sorted by expert,
    expert e has rows offsets[e] to offsets[e + 1], in the order of the pairs, and rows gives each one's token (-1 behind the
    last expert's).  They are what gemm_grouped, gemm_w4 and moe_combine take."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).moe_route(logits, k, normalize)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_moe_route")
    T, E = _dims(logits, "logits", 2)
    k = _integer(k, "k")
    with _on(logits, "logits", stream):
        torch = _pg._torch()
        dev, e = logits.device, _types(logits, "logits")
        _pg._need(logits, "logits", (logits.dtype,), (T, E), dev)
        lib = _pg.load()
        if not 1 <= k <= 32 or k > E:
            raise ValueError(f"k is {k}, expected 1 to {min(E, 32)}")
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)      # noqa: E731
        experts, offsets, slots, rows = new(T, k), new(E + 1), new(T, k), new(T * k)
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        bytes_ = lib.sk_moe_route_work_bytes(T, E)
        work = new(bytes_ // 4) if bytes_ else None
        _run("sk_moe_route", logits.data_ptr(), e, int(bool(normalize)), experts.data_ptr(), weights.data_ptr(),
             offsets.data_ptr(), slots.data_ptr(), rows.data_ptr(), _pg._ptr(work), T, E, k, _pg._stream(logits, None))
    return experts, weights, offsets, slots, rows


def moe_route_backward(dweights, logits, experts, weights, *, normalize=True, stream=None):
    """The logits' gradient [T, E] (of the logits' type), given the gradient dweights (fp32 [T, k]) of moe_route's
    weights and its experts and weights."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).moe_route_backward(dweights, logits, experts, weights, normalize)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_moe_route_backward")
    T, E = _dims(logits, "logits", 2)
    k = _dims(dweights, "dweights", 2)[1]
    with _on(logits, "logits", stream):
        torch = _pg._torch()
        dev, e = logits.device, _types(logits, "logits")
        _pg._need(logits, "logits", (logits.dtype,), (T, E), dev)
        _pg._need(dweights, "dweights", (torch.float32,), (T, k), dev)
        _pg._need(weights, "weights", (torch.float32,), (T, k), dev)
        _whole(experts, "experts", (T, k), dev)
        out = torch.empty_like(logits)
        _run("sk_moe_route_backward", dweights.data_ptr(), logits.data_ptr(), e, int(bool(normalize)), experts.data_ptr(),
             weights.data_ptr(), out.data_ptr(), T, E, k, _pg._stream(logits, None))
    return out


def moe_combine(y, slots, weights=None, *, stream=None):
    """out[t] = sum over j of weights[t, j] * y[slots[t, j]]: y [R, D] (bf16, fp16 or fp32), slots int32 [T, k] (a slot
    outside of 0 to R - 1 is none), weights fp32 [T, k] or None for 1; returns out [T, D] of y's type."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).moe_combine(y, slots, weights)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_moe_combine")
    R, D = _dims(y, "y", 2)
    T, k = _dims(slots, "slots", 2)
    with _on(y, "y", stream):
        torch = _pg._torch()
        dev, e = y.device, _types(y, "y")
        _pg._need(y, "y", (y.dtype,), (R, D), dev)
        _whole(slots, "slots", (T, k), dev)
        _optional(weights, "weights", (torch.float32,), (T, k), dev)
        out = torch.empty((T, D), dtype=y.dtype, device=dev)
        _run("sk_moe_combine", y.data_ptr(), e, slots.data_ptr(), _pg._ptr(weights), out.data_ptr(), T, k, R, D,
             _pg._stream(y, None))
    return out


def moe_combine_backward(dout, y, slots, weights=None, *, offsets=None, stream=None):
    """Gradients of moe_combine: (dy, dweights), dweights None without weights.  No two pairs may share a slot
    (moe_route's do not).  Rows of dy that no slot names are zeros; with moe_route's offsets, which say where those lie, only
    they are cleared and not all of dy first."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).moe_combine_backward(dout, y, slots, weights, offsets)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_moe_combine_backward")
    R, D = _dims(y, "y", 2)
    T, k = _dims(slots, "slots", 2)
    with _on(y, "y", stream):
        torch = _pg._torch()
        dev, e = y.device, _types(y, "y")
        _pg._need(y, "y", (y.dtype,), (R, D), dev)
        _pg._need(dout, "dout", (y.dtype,), (T, D), dev)
        _whole(slots, "slots", (T, k), dev)
        _optional(weights, "weights", (torch.float32,), (T, k), dev)
        E = 0
        if offsets is not None:
            E = _dims(offsets, "offsets", 1)[0] - 1
            _whole(offsets, "offsets", (E + 1,), dev)
        dy = torch.empty_like(y)
        dw = None if weights is None else torch.empty_like(weights)
        _run("sk_moe_combine_backward", dout.data_ptr(), y.data_ptr(), e, slots.data_ptr(), _pg._ptr(weights),
             _pg._ptr(offsets), dy.data_ptr(), _pg._ptr(dw), T, k, R, D, E, _pg._stream(y, None))
    return dy, dw


# ---------------------------------------------------------------- products grouped by expert

def _groups(A, offsets, rows, E, dev):
    """Rows of the grouped product: rows' length, or A's."""
    _whole(offsets, "offsets", (E + 1,), dev)
    if rows is None:
        return A.shape[0]
    R = _dims(rows, "rows", 1)[0]
    _whole(rows, "rows", (R,), dev)
    return R


def _result(out, name, shape, dtype, dev):
    if out is None:
        return _pg._torch().empty(shape, dtype=dtype, device=dev), 1
    _pg._need(out, name, (dtype,), shape, dev)
    return out, 0


def gemm_grouped(A, B, offsets, bias=None, *, rows=None, out=None, stream=None):
    """C[r] = A[rows[r]] . B[e]^T (+ bias[e]) for the rows r = offsets[e] .. offsets[e + 1] - 1 of each expert e; returns C
    [R, N].  A [T, K] and B [E, N, K] are bf16 or fp16 (K a multiple of 8), bias [E, N] of the same type, offsets int32
    [E + 1] and rows int32 [R] as moe_route gives them; without rows, A's own rows lie by expert and R = T.

    The group sizes are read on the device: the call neither waits for them nor depends on them otherwise.  Rows of C behind the
    last expert's are zeros, or in an `out` given by the caller are left as they were."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).gemm_grouped(A, B, offsets, bias, rows, out)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_gemm_grouped")
    T, K = _dims(A, "A", 2)
    E, N, _ = _dims(B, "B", 3)
    with _on(A, "A", stream):
        dev, e = A.device, _types(A, "A", full=False)
        t = (A.dtype,)
        _pg._need(A, "A", t, (T, K), dev)
        _pg._need(B, "B", t, (E, N, K), dev)
        _optional(bias, "bias", t, (E, N), dev)
        R = _groups(A, offsets, rows, E, dev)
        C, zero = _result(out, "out", (R, N), A.dtype, dev)
        _run("sk_gemm_grouped", A.data_ptr(), B.data_ptr(), e, offsets.data_ptr(), _pg._ptr(rows), _pg._ptr(bias),
             C.data_ptr(), R, T, E, N, K, zero, _pg._stream(A, None))
    return C


def gemm_grouped_backward(dC, A, B, offsets, *, rows=None, need_dA=True, need_dB=True, need_dbias=True, stream=None):
    """Gradients of gemm_grouped: (dA, dB, dbias), None where not asked for.  dC is [R, N] of A's type (N, too, a
    multiple of 8, and at most 2^21).  dA [R, K] has a row for each row of the product (zeros behind the last expert's): with rows,
    moe_combine(dA, slots) adds a token's up.  dB [E, N, K] and dbias [E, N] are zeros for an expert without rows."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).gemm_grouped_backward(dC, A, B, offsets, rows, need_dA, need_dB, need_dbias)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_gemm_grouped_backward")
    T, K = _dims(A, "A", 2)
    E, N, _ = _dims(B, "B", 3)
    with _on(A, "A", stream):
        torch = _pg._torch()
        dev, e = A.device, _types(A, "A", full=False)
        t = (A.dtype,)
        _pg._need(A, "A", t, (T, K), dev)
        _pg._need(B, "B", t, (E, N, K), dev)
        R = _groups(A, offsets, rows, E, dev)
        _pg._need(dC, "dC", t, (R, N), dev)
        if not (need_dA or need_dB or need_dbias):
            return None, None, None
        dA = torch.empty((R, K), dtype=A.dtype, device=dev) if need_dA else None
        dB = torch.empty_like(B) if need_dB else None
        db = torch.empty((E, N), dtype=A.dtype, device=dev) if need_dbias else None
        _run("sk_gemm_grouped_backward", dC.data_ptr(), A.data_ptr(), B.data_ptr(), e, offsets.data_ptr(),
             _pg._ptr(rows), _pg._ptr(dA), _pg._ptr(dB), _pg._ptr(db), R, T, E, N, K, _pg._stream(A, None))
    return dA, dB, db


# ---------------------------------------------------------------- 4-bit weights

def quantize_w4(w, group=128, *, zero=False, dtype=None, stream=None):
    """4-bit codes of a weight w [N, K] or, one for each expert, [E, N, K] (bf16, fp16 or fp32), with a scale for each
    `group` (32, 64 or 128; K is a multiple) of elements along a row: (q, scale, zero), w about scale * (code - zero).

    q uint8 [..., N, K / 2] (the even element in the low half of a byte); scale [..., K / group, N] of type `dtype` (bf16 or
    fp16; None: w's own, bf16 for an fp32 w).  zero=False: scale = max|w| / 7 and codes around 8, None is returned
    for zero; zero=True: uint8 zero points [..., K / group, N], scale = (max(w, 0) - min(w, 0)) / 15.  A group that holds an
    infinity or a NaN has a NaN scale."""
    if stream is None:
        torch = _pg._torch()
        half = dtype is torch.float16 or (dtype is None and getattr(w, "dtype", None) is torch.float16)
        if half or dtype is None or dtype is torch.bfloat16:
            got = (_pg._NATIVE or _pg._native()).quantize_w4(w, group, zero, half)
            if got.__class__ is tuple:
                return got
            if got is not None:
                raise _pg.SkError(got, "sk_quantize_w4")
    shape = _dims(w, "w", (2, 3))
    group = _integer(group, "group")
    with _on(w, "w", stream):
        torch = _pg._torch()
        dev, e = w.device, _types(w, "w")
        _pg._need(w, "w", (w.dtype,), shape, dev)
        if dtype is None:
            dtype = torch.bfloat16 if w.dtype == torch.float32 else w.dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"dtype is {dtype}, expected bfloat16 or float16")
        lead, (N, K) = tuple(shape[:-2]), shape[-2:]
        if group not in (32, 64, 128) or K % group:
            raise ValueError(f"group is {group}, expected 32, 64 or 128 and a divisor of {K}")
        q = torch.empty((*lead, N, K // 2), dtype=torch.uint8, device=dev)
        scale = torch.empty((*lead, K // group, N), dtype=dtype, device=dev)
        z = torch.empty(scale.shape, dtype=torch.uint8, device=dev) if zero else None
        _run("sk_quantize_w4", w.data_ptr(), e, q.data_ptr(), scale.data_ptr(), 0 if dtype == torch.bfloat16 else 2,
             _pg._ptr(z), shape[0] if lead else 1, N, K, group, _pg._stream(w, None))
    return q, scale, z


def _codes(q, scale, zero, dev):
    """(lead dimensions, N, K, group) of 4-bit codes with their scales and zero points."""
    shape = _dims(q, "q", (2, 3))
    lead, N, K = tuple(shape[:-2]), shape[-2], 2 * shape[-1]
    _pg._need(q, "q", (_pg._torch().uint8,), shape, dev)
    groups = _dims(scale, "scale", len(shape))[-2]
    if groups < 1 or K % groups or K // groups not in (32, 64, 128):
        raise ValueError(f"scale has {groups} groups for K = {K}, expected groups of 32, 64 or 128")
    _pg._need(scale, "scale", (scale.dtype,), (*lead, groups, N), dev)
    _optional(zero, "zero", (_pg._torch().uint8,), (*lead, groups, N), dev)
    return lead, N, K, K // groups


def dequantize_w4(q, scale, zero=None, *, stream=None):
    """The values scale * (code - zero) of quantize_w4's outputs, of the scale's type: [N, K] or [E, N, K]."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).dequantize_w4(q, scale, zero)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_dequantize_w4")
    with _on(q, "q", stream):
        torch = _pg._torch()
        lead, N, K, group = _codes(q, scale, zero, q.device)
        e = _types(scale, "scale", full=False)
        out = torch.empty((*lead, N, K), dtype=scale.dtype, device=q.device)
        _run("sk_dequantize_w4", q.data_ptr(), scale.data_ptr(), e, _pg._ptr(zero), out.data_ptr(),
             lead[0] if lead else 1, N, K, group, _pg._stream(q, None))
    return out


def gemm_w4(x, q, scale, zero=None, bias=None, *, offsets=None, rows=None, out=None, stream=None):
    """C = x . W^T (+ bias) for few rows of x with the 4-bit weight W = scale * (code - zero) of quantize_w4: x [M, K],
    scale, bias [N] and C [M, N] all bf16 or all fp16.  Sums are fp32; beyond 16 rows the weight is read again for
    every 16 or 32 (with hundreds, dequantize_w4 and an ordinary product are faster).

    With offsets int32 [E + 1], as in gemm_grouped: q [E, N, K / 2], scale and zero [E, K / group, N], bias [E, N], and the rows of
    C by expert; rows int32 [R] chooses x's rows.  Rows of C behind the last expert's are zeros, or in an `out` given by the
    caller left as they were."""
    if stream is None:
        got = (_pg._NATIVE or _pg._native()).gemm_w4(x, q, scale, zero, bias, offsets, rows, out)
        if got.__class__ is not int and got is not None:
            return got
        if got is not None:
            raise _pg.SkError(got, "sk_gemm_w4")
    T, K = _dims(x, "x", 2)
    with _on(x, "x", stream):
        dev, e = x.device, _types(x, "x", full=False)
        t = (x.dtype,)
        _pg._need(x, "x", t, (T, K), dev)
        lead, N, kq, group = _codes(q, scale, zero, dev)
        if kq != K or scale.dtype != x.dtype or bool(lead) != (offsets is not None):
            raise ValueError(f"q {tuple(q.shape)} and scale ({scale.dtype}) do not fit x {tuple(x.shape)} ({x.dtype})"
                             + (" without offsets" if offsets is None else " with offsets"))
        _optional(bias, "bias", t, (*lead, N), dev)
        E, R = 1, T
        if offsets is not None:
            E = lead[0]
            R = _groups(x, offsets, rows, E, dev)
        elif rows is not None:
            raise ValueError("rows come with offsets")
        C, tail = _result(out, "out", (R, N), x.dtype, dev)
        _run("sk_gemm_w4", x.data_ptr(), q.data_ptr(), scale.data_ptr(), _pg._ptr(zero), e, _pg._ptr(offsets),
             _pg._ptr(rows), _pg._ptr(bias), C.data_ptr(), R, T, E, N, K, group, tail, _pg._stream(x, None))
    return C
