"""Paths of the block-scaled calls that need their own sizes or arguments: several 256x256 tiles to a compute unit, as one
stream of k-steps (short K) and dealt singly (long K); launches under a cap; offsets past 32 bits, against plain forms.

Products are of exact inputs (every partial sum is exact in fp32, in any order): equal to the last bit."""

from __future__ import annotations

import pytest
import torch

import block_ref as ref
import persistent_gemm_amd as pg
from test_gpu_fp8_block import _gen, _operands

pytestmark = pytest.mark.gpu


def _values32(q, scale, block):
    """fp32 values of codes: exact for exact operands."""
    return ref.dequantize(q.float(), scale, block).float()


def _check_exact(M, N, K, block, seed, **kw):
    A, B, SA, SB, b = _operands(M, N, K, block, seed, exact=True)
    got = pg.gemm_fp8_block(A.cuda(), B.cuda(), SA.cuda(), SB.cuda(), b.cuda(), **kw).cpu()
    want = _values32(A, SA, "row") @ _values32(B, SB, block).t() + b.float()
    assert torch.equal(got, want.to(torch.bfloat16)), f"{M}x{N}x{K} {block} {kw}"


# 324 tiles and more, which is more than one to a unit.  Blocks of K: streams of 3 to 47 (15 with a scale per row of B),
# odd and even, the last one whole and not; single tiles from there on
@pytest.mark.parametrize("M,N,K,block", [
    (4600, 4400, 880, "tile"), (4401, 4603, 1664, "tile"), (4500, 4360, 2576, "tile"), (4608, 4608, 4224, "tile"),
    (4399, 4612, 6000, "tile"), (4600, 4400, 6016, "tile"), (4600, 4400, 6032, "tile"), (4401, 4500, 6272, "tile"),
    (4600, 4400, 880, "row"), (4401, 4603, 1664, "row"), (4500, 4360, 1904, "row"), (4608, 4608, 1920, "row"),
    (4399, 4612, 1936, "row"), (4600, 4400, 2192, "row"), (8200, 8500, 640, "tile"), (8200, 8500, 656, "row")])
def test_several_tiles_to_a_unit(M, N, K, block):
    _check_exact(M, N, K, block, M + K)


@pytest.mark.parametrize("M,N,K", [(5, 70, 272), (300, 1000, 272), (2100, 2000, 144), (900, 1300, 2064)])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_product_under_a_cap(M, N, K, block):
    for cap in (1, 7, 64, 100000):
        _check_exact(M, N, K, block, cap, grid_cap=cap)


@pytest.mark.parametrize("M,N,K", [(130, 70, 50), (1037, 650, 390), (2050, 130, 200), (100, 2300, 300)])
def test_backward_under_a_cap(M, N, K):
    """dA, dB and dbias of exact inputs: codes of dC are integers times a power of two."""
    g = _gen(M + N + K)
    dC = torch.randint(-7, 8, (M, N), generator=g).float()
    dC[::16] = 7.0      # every block along M and along N holds a 7: its scale is 2^-6, and integers are codes
    dC[:, ::16] = 7.0
    a, b = (torch.randint(-7, 8, s, generator=g).float() for s in ((M, K), (N, K)))
    for x in (a, b):
        x[::16] = 7.0
    At, At_s = pg.quantize_fp8_block(a.cuda(), "row", transpose=True)
    Bt, Bt_s = pg.quantize_fp8_block(b.cuda(), "tile", transpose=True)
    want = dC @ b, dC.t() @ a, dC.sum(0)
    for cap in (0, 1, 7, 64):
        got = pg.gemm_fp8_block_backward(dC.to(torch.bfloat16).cuda(), At, At_s, Bt, Bt_s, grid_cap=cap)
        for name, x, w in zip(("dA", "dB", "dbias"), got, want):
            assert torch.equal(x.cpu(), w.to(torch.bfloat16)), (name, cap)
        only = pg.gemm_fp8_block_backward(dC.to(torch.bfloat16).cuda(), At, At_s, need_dA=False, grid_cap=cap)
        assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])


def test_quantiser_past_32_bits():
    R, C, n = 66000, 33000, 130
    tail = torch.randn(n, C, generator=_gen(7)).to(torch.bfloat16)
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    x[-n:] = tail.cuda()
    q, s, qt, st = pg.quantize_fp8_block(x, transpose="both")
    wq, ws = ref.quantize(tail, "row")
    assert torch.equal(q[-n:].cpu().float().double(), wq) and torch.equal(s[:, -n:].cpu().double(), ws)
    r0 = (R - n) // 128 * 128
    low = torch.zeros(R - r0, C, dtype=torch.bfloat16)
    low[-n:] = tail
    wq, ws = ref.quantize(low.t(), "row")
    assert torch.equal(qt[:, r0:].cpu().float().double(), wq) and torch.equal(st[r0 // 128:].cpu().double(), ws)
    assert (q[:-n].view(torch.uint8) == 0).all()
    del q, s, qt, st
    q, s, qt, st = pg.quantize_fp8_block(x, "tile", transpose="both")
    wq, ws = ref.quantize(low, "tile")
    assert torch.equal(q[r0:].cpu().float().double(), wq) and torch.equal(s[r0 // 128:].cpu().double(), ws)
    wq, ws = ref.quantize(low.t(), "tile")
    assert torch.equal(qt[:, r0:].cpu().float().double(), wq) and torch.equal(st[:, r0 // 128:].cpu().double(), ws)


@pytest.mark.parametrize("block", ["tile", "row"])
def test_product_past_32_bits(block):
    M, N, K = 66000, 33000, 128
    A, B, SA, SB, b = _operands(M, N, K, block, 4, exact=True)
    C = pg.gemm_fp8_block(A.cuda(), B.cuda(), SA.cuda(), SB.cuda(), b.cuda())
    w = _values32(B, SB, block).t()
    for rows in (slice(0, 300), slice(65000, 65400), slice(M - 300, M)):    # (row 65075 is where the bytes pass 2^32)
        want = _values32(A[rows], SA[:, rows], "row") @ w + b.float()
        assert torch.equal(C[rows].cpu(), want.to(torch.bfloat16)), rows


def test_norms_past_32_bits():
    """The last rows' outputs against 64-bit forms; tolerances as in test_gpu_norm.py."""
    from test_gpu_norm import EPS, U, _close
    T, D = 70000, 32000
    g = _gen(8)
    tail = torch.randn(5, D, generator=g).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[-5:] = tail.cuda()
    want, r = ref.rms(tail, w, EPS)
    y, rstd = pg.rms_norm(x, w.cuda(), EPS)
    _close(rstd[-5:], r, 33 * U * r, "rstd")
    _close(y[-5:], want, want.abs() * (40 * U + 2.0 ** -8), "y")
    assert (y[:-5] == 0).all()
    del y
    dx, dw = pg.rms_norm_backward(x, x, w.cuda(), rstd)
    args = (None,) * 7 + (tail, tail, w, rstd[-5:])
    want, bound = ref.norm_backward(*args), ref.norm_backward(*args, sign=-1.0)
    _close(dx[-5:], want["dx"], bound["dx"] * 200 * U + want["dx"].abs() * 2.0 ** -8, "dx")
    assert (dx[:-5] == 0).all()
    # (the zero rows add nothing, exactly)
    _close(dw, want["dnext_weight"], bound["dnext_weight"] * 265 * U + want["dnext_weight"].abs() * 2.0 ** -8, "dweight")


# a size for each kernel: few outputs (short and long K), tiles of 32x32, 64x32, 64x64 (one and two groups), 128x64, 128x128 (four and
# two stages), 256x128, 256x256 (one and several to a unit)
@pytest.mark.parametrize("M,N,K", [(5, 64, 2000), (16, 256, 8192), (16, 8192, 2064), (40, 8200, 640), (500, 700, 400),
                                   (300, 3000, 2064), (1037, 1290, 528), (777, 4099, 300), (1540, 3000, 528),
                                   (3584, 2048, 2064), (2310, 2897, 1000), (4401, 4603, 1664)])
@pytest.mark.parametrize("block", ["tile", "row"])
def test_nan_stays_in_its_rows(M, N, K, block):
    """NaN as a scale of the last block (which ends early, or is followed by blocks that are not there) and as a code."""
    A, B, SA, SB, _ = _operands(M, N, K, block, 5)
    r, c, z = M // 2, N // 3, M - 1
    SA[-1, r] = float("nan")
    A.view(torch.uint8)[z, 1] = 0x7F
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[r] = True
    bad[z] = True
    if block == "tile":
        SB[c // 128, -1] = float("nan")
        bad[:, c // 128 * 128:(c // 128 + 1) * 128] = True
    else:
        SB[-1, c] = float("nan")
        bad[:, c] = True
    got = pg.gemm_fp8_block(A.cuda(), B.cuda(), SA.cuda(), SB.cuda()).cpu()
    assert torch.equal(got.isnan(), bad)
