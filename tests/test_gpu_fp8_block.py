"""The block quantiser, the block-scaled product and its gradients on the GPU, against 64-bit forms on the CPU.

Codes and scales are equal to the last bit.  The product is exact on inputs whose every partial sum is exact;
on random ones |err| <= 2^-8 |C| (the rounding to bf16) + 2^-11 S, S the sum of |terms|: the fp8 matrix
instruction adds its 128 products more coarsely than fp32, up to about 2^-12.8 S on the device, and the fp32 sum over
blocks adds (K / 128 + 3) 2^-24 S, below 2^-15 S for every K here."""

from __future__ import annotations

import pytest
import torch

import block_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _matrix(g, R, C, kind="normal"):
    x = torch.randn(R, C, generator=g) * torch.exp(2 * torch.randn(R, 1, generator=g))
    if kind == "ties":
        # block maxima that are 7 times a power of two give exact scales, and multiples of 1/16 of them exact ties
        x = torch.randint(-224, 225, (R, C), generator=g).float() / 32
        x[:, ::64] = 7.0
    elif kind == "power":
        x = torch.randint(-256, 257, (R, C), generator=g).float()
        x[::3, ::32] = 256.0
    elif kind == "wide":
        x = torch.randn(R, C, generator=g) * torch.exp2(torch.randint(-120, 100, (R, C), generator=g).float())
    elif kind == "tiny":
        x = torch.randn(R, C, generator=g) * 2.0 ** -128
        x[: R // 2] = 0
    return x


def _same_codes(q, want, what):
    got = q.cpu().float().double()
    assert got.shape == want.shape, what
    ok = (got == want) | (got.isnan() & want.isnan())
    assert ok.all(), f"{what}: {int((~ok).sum())} codes differ, first at {(~ok).nonzero()[0].tolist()}"


def _same_scales(s, want, what):
    got = s.cpu().double()
    assert got.shape == want.shape, what
    ok = (got == want) | (got.isnan() & want.isnan())
    assert ok.all(), f"{what}: {int((~ok).sum())} scales differ"


def _check_quantize(x, block, what):
    d = x.cuda()
    wq, ws = ref.quantize(x, block)
    wt, wst = ref.quantize(x.t(), block)
    q, s, qt, st = pg.quantize_fp8_block(d, block, transpose="both")
    for a, b, f in ((q, wq, _same_codes), (s, ws, _same_scales), (qt, wt, _same_codes), (st, wst, _same_scales)):
        f(a, b, what)
    for tr, want in ((False, (wq, ws)), (True, (wt, wst))):
        q1, s1 = pg.quantize_fp8_block(d, block, transpose=tr)
        _same_codes(q1, want[0], what)
        _same_scales(s1, want[1], what)


@pytest.mark.parametrize("kind", ["normal", "ties", "power", "wide", "tiny"])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_values(kind, t, block):
    x = _matrix(_gen(1), 260, 391, kind).to(TYPES[t])
    _check_quantize(x, block, f"{kind} {t} {block}")


@pytest.mark.parametrize("R,C", [(1, 1), (1, 129), (127, 16), (128, 128), (17, 2060), (1025, 24), (130, 1000), (3000, 3003)])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_sizes(R, C, block):
    g = _gen(R * 7 + C)
    for t in TYPES.values():
        _check_quantize(_matrix(g, R, C).to(t), block, f"{R}x{C} {block} {t}")


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_quantize_ties_of_fp32_quotients(t):
    """Maxima all over a binade, so that quotients fall on, and next to, the borders between codes."""
    g = _gen(5)
    top = torch.linspace(1.0, 2.0, 400)[:, None]
    x = top * torch.randint(-64, 65, (400, 128), generator=g).float() / 64
    x[:, 5] = top[:, 0]
    _check_quantize(x.to(TYPES[t]), "row", "ties")


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_infinity_and_nan(t, block):
    x = _matrix(_gen(6), 256, 300).to(TYPES[t])
    x[3, 5] = float("inf")
    x[130, 200] = float("nan")
    if t == "fp32":     # a NaN with every bit of its payload set
        x.view(torch.int32)[200, 290] = 0x7FFFFFFF
    _check_quantize(x, block, f"inf, nan {t} {block}")


def test_quantize_unaligned_view():
    flat = torch.randn(1 + 37 * 130).to(torch.bfloat16).cuda()
    x = flat[1:].view(37, 130)
    q, s = pg.quantize_fp8_block(x)
    q2, s2 = pg.quantize_fp8_block(x.clone())
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_quantize_offsets_past_32_bits():
    R, C = 66000, 33000
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    x[-130:] = torch.randn(130, C, generator=_gen(7)).to(torch.bfloat16).cuda()
    r0 = (R - 130) // 128 * 128
    q, s, qt, st = pg.quantize_fp8_block(x, transpose="both")
    q2, s2, qt2, st2 = pg.quantize_fp8_block(x[r0:].contiguous(), transpose="both")
    assert torch.equal(q[r0:].view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s[:, r0:], s2)
    assert torch.equal(st[r0 // 128:], st2)
    assert torch.equal(qt[:, r0:R].contiguous().view(torch.uint8), qt2[:, :R - r0].contiguous().view(torch.uint8))


# ---------------------------------------------------------------- product

def _operands(M, N, K, block, seed, exact=False):
    g = _gen(seed)
    Kp = ref.up(K, 16)
    kb = ref.up(Kp, 128) // 128
    sb = (ref.up(N, 128) // 128, kb) if block == "tile" else (kb, N)
    if exact:
        # products up to 4, scales 1/2, 1, 2: every partial sum is a multiple of 1/4 below 2^24
        A = torch.randint(-2, 3, (M, Kp), generator=g).float()
        B = torch.randint(-2, 3, (N, Kp), generator=g).float()
        SA = torch.exp2(torch.randint(-1, 2, (kb, M), generator=g).float())
        SB = torch.exp2(torch.randint(-1, 2, sb, generator=g).float())
        bias = torch.randint(-8, 9, (N,), generator=g).float()
    else:
        A = (torch.randn(M, Kp, generator=g) * 100).clamp(-448, 448)
        B = (torch.randn(N, Kp, generator=g) * 100).clamp(-448, 448)
        SA = torch.exp(torch.randn(kb, M, generator=g)) / 448
        SB = torch.exp(torch.randn(*sb, generator=g)) / 448
        bias = torch.randn(N, generator=g)
    A[:, K:] = 0
    B[:, K:] = 0
    return A.to(ref.E4M3), B.to(ref.E4M3), SA, SB, bias.to(torch.bfloat16)


def _check_gemm(M, N, K, block, exact, seed=0, bias=True, **kw):
    A, B, SA, SB, b = _operands(M, N, K, block, seed, exact)
    got = pg.gemm_fp8_block(A.cuda(), B.cuda(), SA.cuda(), SB.cuda(), b.cuda() if bias else None, **kw).cpu()
    a64, b64 = ref.dequantize(A.float(), SA, "row"), ref.dequantize(B.float(), SB, block)
    want = a64 @ b64.t() + (b.double() if bias else 0.0)
    what = f"{M}x{N}x{K} {block} {kw}"
    if exact:
        assert torch.equal(got, want.to(torch.bfloat16)), what
    else:
        S = a64.abs() @ b64.abs().t() + (b.double().abs() if bias else 0.0)
        err = (got.double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -11 * S)
        assert (err <= 0).all(), f"{what}: off by {err.max().item()} more than allowed"


# every kernel: few outputs (short and long K), tiles of 32x32, 64x32, 64x64 (one and two groups of waves), 128x64, 128x128 (two and four stages), 256x128
# and 256x256 (one and several to a workgroup, k-steps even and odd in number), whole and ragged in each dimension
SIZES = [(1, 1, 16), (1, 64, 128), (1, 4096, 4096), (7, 100, 48), (16, 512, 1040), (17, 130, 2064), (32, 96, 256),
         (33, 999, 144), (64, 640, 1000), (65, 63, 16), (100, 100, 2060), (256, 256, 512), (200, 1000, 400),
         (1000, 1500, 272), (777, 4099, 300), (1540, 3000, 528), (4096, 4096, 128), (3000, 4100, 2060),
         (500, 700, 400), (40, 8200, 640), (300, 3000, 2064), (290, 2999, 4100), (2304, 2900, 272), (2310, 2897, 1000),
         (1500, 3100, 300), (16, 8192, 2064), (31, 8300, 400), (1037, 1290, 528), (1100, 1920, 300), (2048, 2048, 400), (200, 300, 1520),
         (130, 250, 4112), (300, 330, 1000), (4200, 4400, 400), (4100, 4501, 300), (8300, 2100, 656), (8200, 8300, 272),
         (2304, 2900, 2064), (2310, 2897, 2100), (2200, 4096, 1040), (2201, 4099, 1040)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("block", ["tile", "row"])
def test_gemm_exact(M, N, K, block):
    _check_gemm(M, N, K, block, True, seed=M + N + K)


@pytest.mark.parametrize("M,N,K", [(1, 100, 3000), (16, 256, 8192), (40, 200, 1000), (130, 190, 4000), (1000, 1500, 700),
                                   (4000, 4096, 600), (500, 700, 5000), (300, 3000, 4096), (2304, 2900, 700), (16, 8192, 8192)])
@pytest.mark.parametrize("block", ["tile", "row"])
def test_gemm_random(M, N, K, block):
    _check_gemm(M, N, K, block, False, seed=K, bias=M % 2 == 0)


@pytest.mark.parametrize("M,N,K", [(5, 70, 272), (300, 1000, 272), (2100, 2000, 144)])
def test_gemm_grid_cap(M, N, K):
    for cap in (1, 7, 64):
        _check_gemm(M, N, K, "tile", True, seed=cap, grid_cap=cap)


def test_gemm_nan_scale_stays_in_its_rows():
    A, B, SA, SB, _ = _operands(300, 260, 400, "tile", 3)
    SA[1, 77] = float("nan")
    SB[1, 2] = float("nan")
    got = pg.gemm_fp8_block(A.cuda(), B.cuda(), SA.cuda(), SB.cuda()).cpu()
    bad = torch.zeros(300, 260, dtype=torch.bool)
    bad[77] = True
    bad[:, 128:256] = True
    assert torch.equal(got.isnan(), bad)


def test_gemm_offsets_past_32_bits():
    M, N, K = 66000, 33000, 128
    A, B, SA, SB, _ = _operands(M, N, K, "tile", 4)
    A, B, SA, SB = A.cuda(), B.cuda(), SA.cuda(), SB.cuda()
    C = pg.gemm_fp8_block(A, B, SA, SB)
    m0 = M // 256 * 256 - 768
    tail = pg.gemm_fp8_block(A[m0:].contiguous(), B, SA[:, m0:].contiguous(), SB)
    assert torch.equal(C[m0:], tail)


def test_gemm_of_quantised_operands_on_another_stream():
    g = _gen(9)
    x, w = torch.randn(200, 700, generator=g).to(torch.bfloat16), torch.randn(300, 700, generator=g) * 0.02
    xd, wd = x.cuda(), w.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a, sa = pg.quantize_fp8_block(xd)
        b, sb = pg.quantize_fp8_block(wd, "tile")
        got = pg.gemm_fp8_block(a, b, sa, sb)
    side.synchronize()
    a64, b64 = ref.dequantize(a.cpu().float(), sa, "row"), ref.dequantize(b.cpu().float(), sb, "tile")
    want, S = a64 @ b64.t(), a64.abs() @ b64.abs().t()
    assert ((got.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * S).all()
    # and near the unquantised product: each factor is off by at most 2^-4 of itself or half the smallest code
    exact = x.double() @ w.double().t()
    step = (x.abs().double() @ w.abs().double().t()) * (2.0 ** -4 * 2 + 2.0 ** -8)
    floor = 700 * 2.0 ** -10 * (sa.max().item() * w.abs().max().item() + sb.max().item() * x.abs().max().item())
    assert ((got.cpu().double() - exact).abs() <= step + floor + 2.0 ** -8 * exact.abs()).all()


def test_forward_calls_replay_in_a_graph():
    g = _gen(10)
    x = torch.randn(70, 512, generator=g).to(torch.bfloat16).cuda()
    wq, ws = pg.quantize_fp8_block((torch.randn(256, 512, generator=g) * 0.02).cuda(), "tile")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pg.gemm_fp8_block(*_pair(x, wq, ws))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pg.gemm_fp8_block(*_pair(x, wq, ws))
    for k in range(4):
        x.copy_(torch.randn(70, 512, generator=_gen(20 + k)).to(torch.bfloat16))
        eager = pg.gemm_fp8_block(*_pair(x, wq, ws))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k


def _pair(x, wq, ws):
    a, sa = pg.quantize_fp8_block(x)
    return a, wq, sa, ws


# ---------------------------------------------------------------- gradients

@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (16, 64, 64), (130, 70, 50), (129, 257, 300), (300, 1000, 200),
                                   (1037, 2050, 1290), (2048, 2304, 2176), (3000, 3200, 70),
                                   (2050, 130, 200), (100, 2300, 300)])
def test_backward(M, N, K):
    g = _gen(M + N + K)
    dC = (torch.randn(M, N, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(torch.bfloat16)
    a, b = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g) * 0.02
    At, At_s = pg.quantize_fp8_block(a.cuda(), "row", transpose=True)
    Bt, Bt_s = pg.quantize_fp8_block(b.cuda(), "tile", transpose=True)
    dA, dB, db = pg.gemm_fp8_block_backward(dC.cuda(), At, At_s, Bt, Bt_s)
    q, s = ref.quantize(dC, "row")
    along_n = ref.dequantize(q, s, "row")
    q, s = ref.quantize(dC.t(), "row")
    along_m = ref.dequantize(q, s, "row")
    bt = ref.dequantize(Bt.cpu().float(), Bt_s, "tile")
    at = ref.dequantize(At.cpu().float(), At_s, "row")
    for name, got, l, r in (("dA", dA, along_n, bt), ("dB", dB, along_m, at)):
        want, S = l @ r.t(), l.abs() @ r.abs().t()
        err = (got.cpu().double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -11 * S)
        assert (err <= 0).all(), f"{name}: off by {err.max().item()} more than allowed"
    want, S = dC.double().sum(0), dC.double().abs().sum(0)
    # sums of 128 rows (8 + 16 terms deep), then of M / 128: below 60 additions in a chain
    assert ((db.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 60 * 2.0 ** -24 * S).all()
    # the same bits again, and each output alone
    again = pg.gemm_fp8_block_backward(dC.cuda(), At, At_s, Bt, Bt_s)
    assert torch.equal(again[0], dA) and torch.equal(again[1], dB) and torch.equal(again[2], db)
    only = pg.gemm_fp8_block_backward(dC.cuda(), None, None, Bt, Bt_s, need_dB=False, need_dbias=False)
    assert torch.equal(only[0], dA) and only[1] is None and only[2] is None
    only = pg.gemm_fp8_block_backward(dC.cuda(), At, At_s, need_dA=False, need_dbias=False)
    assert torch.equal(only[1], dB)
    only = pg.gemm_fp8_block_backward(dC.cuda(), need_dA=False, need_dB=False)
    assert torch.equal(only[2], db)


def test_backward_refuses_capture():
    dC = torch.randn(64, 64).to(torch.bfloat16).cuda()
    pg.gemm_fp8_block_backward(dC, need_dA=False, need_dB=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(pg.SkError, match="UNSUPPORTED"):
            pg.gemm_fp8_block_backward(dC, need_dA=False, need_dB=False)


# ---------------------------------------------------------------- refusals of the binding

def test_refusals():
    x = torch.randn(32, 64, device="cuda")
    q, s = pg.quantize_fp8_block(x)
    for bad, kind in ((lambda: pg.quantize_fp8_block(x.half()), TypeError),
                      (lambda: pg.quantize_fp8_block(x.t()), ValueError),
                      (lambda: pg.quantize_fp8_block(x, "column"), ValueError),
                      (lambda: pg.quantize_fp8_block(x, transpose="yes"), ValueError),
                      (lambda: pg.quantize_fp8_block(x[0]), ValueError),
                      (lambda: pg.quantize_fp8_block(x[:0]), pg.SkError),
                      (lambda: pg.gemm_fp8_block(q, q, s, s[:, :5]), ValueError),
                      (lambda: pg.gemm_fp8_block(q, q[:, :48].contiguous(), s, s), ValueError),
                      (lambda: pg.gemm_fp8_block(q, q, s, s.double()), TypeError),
                      (lambda: pg.gemm_fp8_block(q, q, s.cpu(), s), ValueError),
                      (lambda: pg.gemm_fp8_block(q[:, :8].contiguous(), q[:, :8].contiguous(), s, s), pg.SkError),
                      (lambda: pg.gemm_fp8_block_backward(x), TypeError),
                      (lambda: pg.gemm_fp8_block_backward(x.bfloat16()), ValueError)):
        with pytest.raises(kind):
            bad()
