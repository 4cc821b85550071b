"""Codes of blocks whose scale is among the smallest normal numbers: a quotient next to the border of two codes differs
from it by less than the smallest number of its type there.  Against 64-bit forms, to the last bit."""

from __future__ import annotations

import pytest
import torch

import block_ref as ref
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu


def _next_to_borders():
    """fp32 rows of 128: each starts with 448 s, for scales s = 2^e (1 + k 2^-23) from 2^-126 on; then the borders
    between the codes (two codes' mean, times 2^e and times s), and their neighbours."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(ref.E4M3).double()
    borders = (codes[1:] + codes[:-1]) / 2
    g = torch.Generator().manual_seed(11)
    rows = []
    for e in list(range(-126, -88)) + [-60, 0, 100]:
        for k in [0, 1, 2, 3, 101, (1 << 23) - 1] + torch.randint(0, 1 << 23, (4,), generator=g).tolist():
            s = 2.0 ** e * (1 + k * 2.0 ** -23)
            for unit, first in ((2.0 ** e, 0), (2.0 ** e, 40), (s, 0), (s, 84)):
                b = (borders[first:first + 42] * unit).float()
                b = b[b.abs() <= 448 * s]
                near = torch.cat([b, torch.nextafter(b, torch.tensor(0.0)), -torch.nextafter(b, torch.tensor(1e38))])
                row = torch.zeros(128)
                row[:len(near)] = near.clamp(-448 * s, 448 * s)
                row[127] = 448 * s
                rows.append(row)
    return torch.stack(rows)


def _equal(got, want, what):
    got = got.cpu().float().double()
    assert got.shape == want.shape
    bad = got != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


def test_rows_and_columns():
    x = _next_to_borders()
    q, s = ref.quantize(x, "row")
    got = pg.quantize_fp8_block(x.cuda())
    _equal(got[1], s, "scales")
    _equal(got[0], q, "codes")
    # along the rows of the transpose, with the plain form beside them
    qt, st = pg.quantize_fp8_block(x.t().contiguous().cuda(), transpose="both")[2:]
    _equal(st, s, "scales of the transpose")
    _equal(qt[:, :128], q, "codes of the transpose")


def test_many_tiles():
    """The same, often enough that a thread takes more rows."""
    x = _next_to_borders()
    q, s = ref.quantize(x, "row")
    n = 45
    got = pg.quantize_fp8_block(x.repeat(1, n).cuda())
    _equal(got[1], s.repeat(n, 1), "scales")
    _equal(got[0], q.repeat(1, n), "codes")
    for transpose in (True, "both"):
        qt, st = pg.quantize_fp8_block(x.t().repeat(n, 1).cuda(), transpose=transpose)[-2:]
        _equal(st, s.repeat(n, 1), "scales of the transpose")
        _equal(qt, q.repeat(1, n), "codes of the transpose")


def test_tiles():
    x = _next_to_borders()
    for first in list(range(4, 60, 4)) + list(range(84, 400, 40)):      # a row and 127 quiet ones
        t = torch.zeros(128, 128)
        t[7] = x[first + 2]
        q, s = ref.quantize(t, "tile")
        got = pg.quantize_fp8_block(t.cuda(), "tile", transpose="both")
        _equal(got[1], s, "scale")
        _equal(got[0], q, "codes")
        _equal(got[2], q.t(), "codes of the transpose")


def test_bf16():
    """All 8-bit mantissas of the largest element, with every bf16 next to a border."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(ref.E4M3).double()
    borders = (codes[1:] + codes[:-1]) / 2
    rows = []
    for e in (-126, -125, -120, -110, -100, 0):
        for m in range(128, 256):
            top = 2.0 ** (e + 8) * m / 128
            near = (borders[:125] * (top / 448)).float().to(torch.bfloat16)
            rows.append(torch.cat([near, near.new_tensor([0.0, -top, top])]))
    x = torch.stack(rows)
    q, s = ref.quantize(x, "row")
    got = pg.quantize_fp8_block(x.cuda())
    _equal(got[1], s, "scales")
    _equal(got[0], q, "codes")


@pytest.mark.parametrize("T,D", [(50, 256), (9, 4096)])
def test_norm_of_tiny_weights(T, D):
    """The norm's codes are those of its fp32 output."""
    g = torch.Generator().manual_seed(12)
    for e in (-126, -120, -110, -98, -96, -90):
        x = torch.randn(T, D, generator=g).cuda()
        w = (2.0 ** (e + 8) * torch.exp2(-torch.randint(0, 12, (D,), generator=g).float())).cuda()
        y, _ = pg.rms_norm(x, w)
        q, s, _ = pg.rms_norm(x, w, quantize=True)
        wq, ws = ref.quantize(y, "row")
        _equal(s, ws, f"scales {e}")
        _equal(q, wq, f"codes {e}")
