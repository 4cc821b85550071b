"""A layer of experts beside the ordinary call: every tile, other streams and threads, captured graphs, misaligned and strided
tensors, addresses past 32 bits, refusals."""

from __future__ import annotations

import threading

import pytest
import torch

import experts_ref as ref
import test_gpu_experts as plain
import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(seed, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=_gen(seed)) * scale).to(dtype).cuda()


def _offsets(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32).cuda()


# ---------------------------------------------------------------- tiles

# Large tiles, which are cut into 1, 2 and 4 pieces where few are left for the last turn (256 units: 3 x 64 = 192 tiles, 2 x 64 = 128,
# and 5 x 64 = 256 + 64, the last rows fewer than a piece), over ends of rows and columns.
CUT = [([300, 212], 16384), ([300, 212], 16373), ([512], 16384), ([400], 16200), ([1100], 16384), ([1100], 16373), ([130, 0, 1000, 4], 16376),
       ([300, 900], 12289)]


@pytest.mark.parametrize("gather", [0, 90])
@pytest.mark.parametrize("counts,N", CUT)
def test_forward_cut_tiles(counts, N, gather):
    K, R, E = 72, sum(counts), len(counts)
    offsets = _offsets(counts)
    rows = torch.randint(0, gather, (R,), generator=_gen(1)).to(torch.int32).cuda() if gather else None
    A, B, b = _rand(2, gather or R, K), _rand(3, E, N, K), _rand(4, E, N)
    got = pg.gemm_grouped(A, B, offsets, b, rows=rows)
    want, mag = ref.grouped(A, B, offsets, b, rows)
    ref.assert_near(got, want, ref.rounding(want, BF) * 1.001 + mag * (K + 1) * ref.STEP32)


@pytest.mark.parametrize("counts,K", [(c, n // 8 * 8) for c, n in CUT])
def test_row_gradient_cut_tiles(counts, K):
    N, R, E = 72, sum(counts) + 5, len(counts)
    offsets = _offsets(counts)
    A, B, d = torch.empty(R, K, dtype=HF, device="cuda"), _rand(3, E, N, K, dtype=HF), _rand(4, R, N, dtype=HF)
    got = pg.gemm_grouped_backward(d, A, B, offsets, need_dB=False, need_dbias=False)[0]
    want = torch.zeros(R, K, dtype=torch.float64)
    mag = torch.zeros_like(want)
    for e, lo, hi in ref.spans(offsets, R):
        x, b = d[lo:hi].double().cpu(), B[e].double().cpu()
        want[lo:hi], mag[lo:hi] = x @ b, x.abs() @ b.abs()
    ref.assert_near(got, want, ref.rounding(want, HF) * 1.001 + mag * (N + 1) * ref.STEP32)


# Each size of tile (rows x columns of the output; 256 units) in each direction, its ends within a tile.
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,N,K", [
    ([33, 0, 200, 7], 400, 136),                 # 32 x 128
    ([1000, 0, 1061], 520, 264),                 # 64 x 128
    ([1000, 63, 1500], 777, 136),                # 128 x 128
    ([2, 40, 0, 90, 500, 31] * 6, 1100, 72),     # 128 x 128, more experts than full tiles
    ([700, 300, 600], 4099, 200),                # 256 x 256, whole and cut
])
def test_forward_tiles(counts, N, K, dtype):
    plain._check_grouped(counts, N, K, dtype, bias=True, gather=77, tail=3)
    plain._check_grouped(counts, N, K, dtype)


@pytest.mark.parametrize("gather", [0, 77])
@pytest.mark.parametrize("counts,N,K,dtype", [
    ([33, 0, 200, 7], 136, 400, BF), ([1000, 0, 1061], 264, 520, HF), ([1000, 63, 1500], 136, 776, BF),
    ([2, 40, 0, 90, 500, 31] * 6, 72, 1096, HF), ([700, 300, 600], 200, 4104, BF),
    ([300, 0, 513], 2056, 1544, BF), ([65, 1, 130], 1800, 2312, HF),        # dB in tiles of 256 x 256
])
def test_backward_tiles(counts, N, K, dtype, gather):
    plain._check_grouped_backward(counts, N, K, dtype, gather=gather, tail=4)


def test_not_finite_values_stay_in_their_rows():
    """An infinity or a NaN of one row or expert is in no other's outputs (rows share tiles and k-steps)."""
    counts, N, K = [3, 5, 0, 70], 40, 72
    R, offsets = sum(counts), _offsets(counts)
    A, B, d = _rand(1, R, K), _rand(2, 4, N, K), _rand(3, R, N)
    A[2, 71], A[3, 0], A[10, 5], B[2, 7, 7], d[7, 39] = float("nan"), float("inf"), float("-inf"), float("nan"), float("inf")
    C = pg.gemm_grouped(A, B, offsets).cpu()
    bad = ~torch.isfinite(C).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [2, 3, 10]
    assert torch.isnan(C[2]).all() and not torch.isfinite(C[[2, 3, 10]]).any()
    dA, dB, db = (t.cpu() for t in pg.gemm_grouped_backward(d, A, B, offsets))
    assert (~torch.isfinite(dA).all(dim=1)).nonzero().flatten().tolist() == [7]
    bad = ~torch.isfinite(dB)
    assert not bad[2].any()
    assert bad[0].nonzero()[:, 1].unique().tolist() == [71] and bad[3].nonzero()[:, 1].unique().tolist() == [5]
    assert bad[1][39].all() and bad[1][:39].nonzero()[:, 1].unique().tolist() == [0]
    assert (~torch.isfinite(db)).nonzero().tolist() == [[1, 39]]


# ---------------------------------------------------------------- the layer as it is used

class Layer:
    """A layer's training step and its serving step on fixed tensors; x and dout may be changed between calls."""

    def __init__(self, T, D, H, E, k, dtype=BF, seed=0):
        self.k = k
        self.x, self.dout = _rand(seed, T, D, dtype=dtype), _rand(seed + 1, T, D, dtype=dtype)
        self.router, self.all = _rand(seed + 2, 1, E, D, dtype=dtype, scale=D ** -0.5), _offsets([T])
        self.W1, self.b1 = _rand(seed + 3, E, H, D, dtype=dtype, scale=D ** -0.5), _rand(seed + 4, E, H, dtype=dtype)
        self.W2 = _rand(seed + 5, E, D, H, dtype=dtype, scale=H ** -0.5)
        self.q1, self.q2 = pg.quantize_w4(self.W1, 64, zero=True), pg.quantize_w4(self.W2, 32)

    def train(self, **kw):
        logits = pg.gemm_grouped(self.x, self.router, self.all, **kw)
        ids, w, offsets, slots, rows = pg.moe_route(logits, self.k, **kw)
        r = torch.relu(pg.gemm_grouped(self.x, self.W1, offsets, self.b1, rows=rows, **kw))
        y = pg.gemm_grouped(r, self.W2, offsets, **kw)
        out = pg.moe_combine(y, slots, w, **kw)
        dy, dw = pg.moe_combine_backward(self.dout, y, slots, w, offsets=offsets, **kw)
        dr, dW2, _ = pg.gemm_grouped_backward(dy, r, self.W2, offsets, need_dbias=False, **kw)
        dxr, dW1, db1 = pg.gemm_grouped_backward(dr * (r > 0), self.x, self.W1, offsets, rows=rows, **kw)
        dl = pg.moe_route_backward(dw, logits, ids, w, **kw)
        return [ids, w, offsets, slots, rows, out, dW1, db1, dW2, pg.moe_combine(dxr, slots, **kw), dl]

    def serve(self, **kw):
        logits = pg.gemm_grouped(self.x, self.router, self.all, **kw)
        _, w, offsets, slots, rows = pg.moe_route(logits, self.k, **kw)
        r = torch.relu(pg.gemm_w4(self.x, *self.q1, self.b1, offsets=offsets, rows=rows, **kw))
        return [pg.moe_combine(pg.gemm_w4(r, *self.q2, offsets=offsets, **kw), slots, w, **kw)]

    def change(self, seed):
        self.x.copy_(_rand(seed, *self.x.shape, dtype=self.x.dtype))
        self.dout.copy_(_rand(seed + 1, *self.x.shape, dtype=self.x.dtype))


def _same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("T,D,H,E,k", [(1, 64, 96, 8, 2), (70, 192, 128, 16, 4), (600, 256, 192, 5, 2)])
def test_captured_and_replayed(T, D, H, E, k):
    layer = Layer(T, D, H, E, k)
    layer.train(), layer.serve()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.train() + layer.serve()
    for i in range(4):
        layer.change(100 + 10 * i)
        want = [t.clone() for t in layer.train() + layer.serve()]
        for t in got:
            t.view(torch.uint8).fill_(0xa5)
        graph.replay()
        torch.cuda.synchronize()
        _same(got, want)


def test_two_graphs_and_streams_at_once():
    """Graphs of two layers, and eager calls of a third, on streams of their own at one time."""
    layers = [Layer(300, 128, 192, 8, 2, seed=20 * i) for i in range(3)]
    want = [[t.clone() for t in x.train() + x.serve()] for x in layers]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in layers[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.train() + x.serve())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = layers[2].train() + layers[2].serve()
        torch.cuda.synchronize()
        for a, b in zip(outs + [eager], want):
            _same(a, b)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_stream_argument(dtype):
    """A stream given as such or as a handle: the same bits as on the current one, and the outputs are its own."""
    layer = Layer(130, 128, 128, 9, 3, dtype=dtype)
    want = [t.clone() for t in layer.train() + layer.serve()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):           # (torch's own operations between the calls have to be on it too)
        for kw in (dict(stream=s), dict(stream=s.cuda_stream), dict(stream=None)):
            _same(layer.train(**kw) + layer.serve(**kw), want)
    logits = _rand(9, 40, 16, dtype=FP)
    torch.cuda.synchronize()
    got = pg.moe_route(logits, 3, stream=s)
    s.synchronize()
    _same(got, pg.moe_route(logits, 3))


def test_host_threads():
    layers = [Layer(100 + 60 * i, 128, 128, 8, 2, seed=30 * i) for i in range(3)]
    want = [[t.clone() for t in x.train() + x.serve()] for x in layers]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got = layers[i].train() + layers[i].serve()
                    s.synchronize()
                    _same(got, want[i])
        except BaseException as e:      # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad, bad


def test_calls_repeat():
    layer = Layer(900, 256, 320, 12, 4)
    first = [t.clone() for t in layer.train() + layer.serve()]
    for _ in range(3):
        _same(layer.train() + layer.serve(), first)


# ---------------------------------------------------------------- tensors that are not as usual

def _shifted(t, by=1):
    """The same values at an address `by` elements further on."""
    big = torch.zeros(t.numel() + 16, dtype=t.dtype, device=t.device)
    v = big[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def test_elementwise_alignment():
    """What need only be aligned to its elements gives the same bits there."""
    layer = Layer(37, 128, 192, 6, 2)
    x, o = layer.x, torch.tensor([0, 3, 20, 20, 30, 37, 37], dtype=torch.int32).cuda()
    r = torch.arange(36, -1, -1, dtype=torch.int32).cuda()
    want = pg.gemm_grouped(x, layer.W1, o, layer.b1, rows=r)
    out = _shifted(torch.zeros_like(want))
    got = pg.gemm_grouped(x, layer.W1, _shifted(o), _shifted(layer.b1), rows=_shifted(r), out=out)
    assert got is out and torch.equal(got, want)
    q, s, z = layer.q1
    # (with other alignment the waves take other steps, and so another order of sums: against 64 bits, each addition of the
    # 2 K terms, the groups' products and the bias off by at most a step)
    far = (2 * 64 + 2 + 8) * ref.STEP32
    got = pg.gemm_w4(x, q, _shifted(s), _shifted(z), _shifted(layer.b1), offsets=_shifted(o), rows=_shifted(r)).cpu()
    for e, lo, hi in ref.spans(o, 37):
        if lo < hi:
            want, mag = ref.w4(x[r[lo:hi].long()], q[e], s[e], z[e], layer.b1[e], 64)
            ref.assert_near(got[lo:hi], want, ref.rounding(want, BF) * 1.001 + mag * far)
    want, mag = ref.w4(x[:5], q[1], s[1], z[1], None, 64)
    ref.assert_near(pg.gemm_w4(x[:5], q[1], _shifted(s[1]), _shifted(z[1])), want, ref.rounding(want, BF) * 1.001 + mag * far)
    for dtype in (BF, HF, FP):
        logits = _rand(1, 70, 37, dtype=dtype)
        a, b = pg.moe_route(logits, 4, normalize=False), pg.moe_route(_shifted(logits), 4, normalize=False)
        _same(a, b)
        dw = _rand(2, 70, 4, dtype=FP)
        assert torch.equal(pg.moe_route_backward(dw, logits, a[0], a[1], normalize=False),
                           pg.moe_route_backward(_shifted(dw), _shifted(logits), _shifted(a[0]), _shifted(a[1]), normalize=False))
        logits = _rand(1, 70, 64, dtype=dtype)          # E a multiple of a lane's logits, their address not
        _same(pg.moe_route(logits, 4), pg.moe_route(_shifted(logits), 4))
        y, dout = _rand(3, 280, 72, dtype=dtype), _rand(4, 70, 72, dtype=dtype)
        assert torch.equal(pg.moe_combine(y, a[3], a[1]), pg.moe_combine(_shifted(y), _shifted(a[3]), _shifted(a[1])))
        _same(pg.moe_combine_backward(dout, y, a[3], a[1], offsets=a[2]),
              pg.moe_combine_backward(_shifted(dout), _shifted(y), _shifted(a[3]), _shifted(a[1]), offsets=_shifted(a[2])))
        w = _rand(5, 33, 256, dtype=dtype)
        _same(pg.quantize_w4(w, 64, zero=True), pg.quantize_w4(_shifted(w), 64, zero=True))
        q, s, z = pg.quantize_w4(w, 64, zero=True)
        assert torch.equal(pg.dequantize_w4(q, s, z), pg.dequantize_w4(q, _shifted(s), _shifted(z)))


def test_refusals():
    x, W, o = _rand(1, 8, 64), _rand(2, 2, 16, 64), _offsets([3, 5])
    q, s, z = pg.quantize_w4(W, 32, zero=True)
    logits = _rand(3, 8, 16, dtype=FP)
    ids, w, offsets, slots, rows = pg.moe_route(logits, 2)
    T, V, S = TypeError, ValueError, pg.SkError
    for err, call in [
        (V, lambda: pg.moe_route(logits.cpu(), 2)), (T, lambda: pg.moe_route(logits.double(), 2)), (V, lambda: pg.moe_route(logits, 0)),
        (V, lambda: pg.moe_route(logits, 17)), (V, lambda: pg.moe_route(logits[0], 2)), (V, lambda: pg.moe_route(logits[:, ::2], 2)),
        (V, lambda: pg.moe_route(logits.t(), 2)), (S, lambda: pg.moe_route(logits[:0], 2)), (T, lambda: pg.moe_route([[1.0]], 1)),
        (RuntimeError, lambda: pg.moe_route(logits, 2, normalize=logits)),
        (V, lambda: pg.moe_route_backward(w[:7], logits, ids, w)), (T, lambda: pg.moe_route_backward(w, logits, ids.long(), w)),
        (T, lambda: pg.moe_route_backward(w.half(), logits, ids, w)), (V, lambda: pg.moe_route_backward(w, logits, ids.cpu(), w)),
        (T, lambda: pg.moe_combine(x, slots.long(), w)), (V, lambda: pg.moe_combine(x, slots, w[:7])), (V, lambda: pg.moe_combine(x.t(), slots)),
        (T, lambda: pg.moe_combine(x.double(), slots)), (V, lambda: pg.moe_combine_backward(x[:7], x, slots, w)),
        (T, lambda: pg.moe_combine_backward(x, x, slots, w, offsets=offsets.long())),
        (T, lambda: pg.moe_combine_backward(x.float(), x, slots, w)),
        (T, lambda: pg.gemm_grouped(x.float(), W.float(), o)), (T, lambda: pg.gemm_grouped(x, W.half(), o)), (V, lambda: pg.gemm_grouped(x, W[0], o)),
        (V, lambda: pg.gemm_grouped(x, W[:, :, :56], o)), (V, lambda: pg.gemm_grouped(x, W, o[:2])), (T, lambda: pg.gemm_grouped(x, W, o.long())),
        (V, lambda: pg.gemm_grouped(x, W, o.cpu())), (V, lambda: pg.gemm_grouped(x, W.transpose(1, 2), o)), (T, lambda: pg.gemm_grouped(x, W, None)),
        (V, lambda: pg.gemm_grouped(x, W, o, W[0])), (V, lambda: pg.gemm_grouped(x, W, o, out=x)), (S, lambda: pg.gemm_grouped(x[:, :4].contiguous(), W[:, :, :4].contiguous(), o)),
        (T, lambda: pg.gemm_grouped(x, W, o, rows=rows.long())), (S, lambda: pg.gemm_grouped(_shifted(x), W, o)), (S, lambda: pg.gemm_grouped(x[:0], W, o)),
        (V, lambda: pg.gemm_grouped_backward(x, x, W, o)), (S, lambda: pg.gemm_grouped_backward(x[:, :15].contiguous(), x, W[:, :15].contiguous(), o)),
        (S, lambda: pg.gemm_grouped(x, W, o, out=x.view(-1)[64:192].view(8, 16))),
        (V, lambda: pg.quantize_w4(x, 48)), (V, lambda: pg.quantize_w4(x, 128)), (T, lambda: pg.quantize_w4(x.double(), 32)),
        (V, lambda: pg.quantize_w4(x.t(), 32)), (T, lambda: pg.quantize_w4(x, 32, dtype=FP)), (V, lambda: pg.quantize_w4(x[0], 32)),
        (T, lambda: pg.dequantize_w4(q.int(), s)), (V, lambda: pg.dequantize_w4(q, s[:, :1, :8])), (V, lambda: pg.dequantize_w4(q, s, z[:1])),
        (T, lambda: pg.dequantize_w4(q, s.float())), (T, lambda: pg.gemm_w4(x.float(), q, s, offsets=o)), (V, lambda: pg.gemm_w4(x, q, s)),
        (V, lambda: pg.gemm_w4(x, q[0], s[0], offsets=o)), (V, lambda: pg.gemm_w4(x, q[0], s[0], rows=rows)), (V, lambda: pg.gemm_w4(x.half(), q, s, offsets=o)),
        (V, lambda: pg.gemm_w4(x[:, :32].contiguous(), q, s, offsets=o)), (V, lambda: pg.gemm_w4(x, q, s, offsets=o[:2])),
        (T, lambda: pg.gemm_w4(x, q, s, z.int(), offsets=o)), (V, lambda: pg.gemm_w4(x, q, s, offsets=o, out=x)), (S, lambda: pg.gemm_w4(_shifted(x), q, s, offsets=o)),
    ]:
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()


# ---------------------------------------------------------------- addresses past 32 bits



def test_large_outputs_and_inputs():
    """Tensors of over 4 GiB: rows near their ends against products of those rows alone."""
    R, N, K, E = 70000, 32776, 8, 3
    o = torch.tensor([0, 10, 69000, 70000], dtype=torch.int32).cuda()
    A, B = _rand(1, R, K), _rand(2, E, N, K)
    C = pg.gemm_grouped(A, B, o)
    for a, b, e in ((0, 10, 0), (60000, 60300, 1), (69900, 70000, 2)):
        part = pg.gemm_grouped(A[a:b].contiguous(), B[e:e + 1].contiguous(), torch.tensor([0, b - a], dtype=torch.int32).cuda())
        assert torch.equal(C[a:b], part), a
    dA, dB, _ = pg.gemm_grouped_backward(C, A, B, o, need_dbias=False)
    part = pg.gemm_grouped_backward(C[69000:].contiguous(), A[69000:].contiguous(), B[2:].contiguous(), torch.tensor([0, 1000], dtype=torch.int32).cuda())
    assert torch.equal(dB[2:], part[1])
    ref.assert_near(dA[69990:], C[69990:].double().cpu() @ B[2].double().cpu(), (C[69990:].double().cpu().abs() @ B[2].double().cpu().abs()) * (2.0 ** -8 + N * ref.STEP32))
    # the sum of its rows, and its gradient
    slots = torch.tensor([[0, 69999], [65537, 3], [65535, -1]], dtype=torch.int32).cuda()
    w = _rand(4, 3, 2, dtype=FP)
    out = pg.moe_combine(C, slots, w)
    f = C[slots.clamp(min=0).long()].double()
    want = (f[:, 0] * w[:, :1].double() + f[:, 1] * (w[:, 1:].double() * (slots[:, 1:] >= 0)))
    ref.assert_near(out, want.cpu(), ref.rounding(want.cpu(), BF) * 1.001 + (f.abs().sum(dim=1) * w.abs().amax()).cpu() * 4 * ref.STEP32)
    dy, dw = pg.moe_combine_backward(out, C, slots, w)
    assert torch.equal(dy[69999], (w[0, 1] * out[0].float()).to(BF)) and torch.equal(dy[65537], (w[1, 0] * out[1].float()).to(BF))
    assert torch.equal(dy[65535], (w[2, 0] * out[2].float()).to(BF)) and not dy[65536].any() and not dy[69998].any() and float(dw[2, 1]) == 0


def test_large_weights():
    """Weights of over 4 GiB, in 16 and in 4 bits: the last experts' rows against those experts alone."""
    E, N, K = 40, 8192, 8192
    W = torch.empty(E, N, K, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    o = _offsets([2] * E)
    x = _rand(2, 2 * E, K)
    two = torch.tensor([0, 2], dtype=torch.int32).cuda()
    C = pg.gemm_grouped(x, W, o)
    for e in (0, 15, 16, 32, 39):
        assert torch.equal(C[2 * e:2 * e + 2], pg.gemm_grouped(x[2 * e:2 * e + 2].contiguous(), W[e:e + 1], two)), e
    del C
    q, s, z = pg.quantize_w4(W, 64, zero=True)
    back = pg.dequantize_w4(q, s, z)
    for e in (0, 31, 32, 39):
        _same(pg.quantize_w4(W[e], 64, zero=True), (q[e], s[e], z[e]))
        assert torch.equal(back[e], pg.dequantize_w4(q[e], s[e], z[e])), e
    del W, back
    big = torch.cat([q, q, q, q])           # codes of 5 GiB
    bs, bz = torch.cat([s] * 4), torch.cat([z] * 4)
    x = _rand(3, 4 * E, K)
    C = pg.gemm_w4(x, big, bs, bz, offsets=_offsets([1] * (4 * E)))
    one = torch.tensor([0, 1], dtype=torch.int32).cuda()
    for e in (0, 127, 128, 159):
        assert torch.equal(C[e:e + 1], pg.gemm_w4(x[e:e + 1].contiguous(), q[e % E:e % E + 1], s[e % E:e % E + 1], z[e % E:e % E + 1], offsets=one)), e


def test_long_logits():
    """Logits of over 4 GiB: the choices of the last tokens, and the places of all pairs."""
    T, E = 1200000, 1024
    logits = torch.empty(T, E, dtype=FP, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    ids, w, offsets, slots, rows = pg.moe_route(logits, 2)
    top = logits[-1000:].sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids[-1000:].long(), top.indices[:, :2])
    order = torch.sort(ids.reshape(-1), stable=True).indices
    assert torch.equal(rows.long(), order // 2)
    assert torch.equal(offsets[1:].long(), torch.bincount(ids.reshape(-1).long(), minlength=E).cumsum(0))
    assert torch.equal(slots.reshape(-1)[order].long(), torch.arange(2 * T, device="cuda"))
    d = pg.moe_route_backward(torch.ones_like(w) * torch.tensor([1.0, 0.0], device="cuda"), logits, ids, w)
    tail = pg.moe_route_backward(torch.ones_like(w[-64:]) * torch.tensor([1.0, 0.0], device="cuda"), logits[-64:].contiguous(), ids[-64:].contiguous(), w[-64:].contiguous())
    assert torch.equal(d[-64:], tail)
