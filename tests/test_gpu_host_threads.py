"""Host threads that share a stream, on the GPU: every call's outputs are those of the same call made alone.

The threads go through the C entry points (ctypes gives the interpreter lock up for a call), with sizes
that make the stream's scratch grow in turns."""

from __future__ import annotations

import ctypes
import threading

import pytest
import torch

import persistent_gemm_amd as pg

pytestmark = pytest.mark.gpu


def _block_backward(M, N, K, grid_cap=0):
    g = torch.Generator().manual_seed(M + N + K)
    dC = torch.randn(M, N, generator=g).to(torch.bfloat16).cuda()
    at, at_s = pg.quantize_fp8_block(torch.randn(M, K, generator=g).cuda(), transpose=True)
    bt, bt_s = pg.quantize_fp8_block(torch.randn(N, K, generator=g).cuda(), "tile", transpose=True)

    def call(stream):
        out = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (N, K), (N,))]
        p = [t.data_ptr() for t in (dC, at, at_s, bt, bt_s, *out)]
        return out, lambda: pg.load().sk_gemm_fp8_block_backward(*p, M, N, K, grid_cap, stream)
    return call


def _bf16_backward(M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    dC, A, B = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((M, N), (M, K), (N, K)))

    def call(stream):
        out = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (N, K), (N,))]
        p = [t.data_ptr() for t in (dC, A, B, *out)]
        return out, lambda: pg.load().sk_gemm_bf16_backward(*p, M, N, K, 0, stream)
    return call


def _norm_backward(T, D):
    g = torch.Generator().manual_seed(T + D)
    dout, h, w = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((T, D), (T, D), (D,)))
    _, rstd = pg.rms_norm(h, w)

    def call(stream):
        out = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((T, D), (T, D), (D,))]
        a = pg._NormGradArgs(elem=0, dout=dout.data_ptr(), h=h.data_ptr(), weight=w.data_ptr(), rstd=rstd.data_ptr(),
                             dx=out[0].data_ptr(), dresidual=out[1].data_ptr(), dweight=out[2].data_ptr(), T=T, D=D,
                             stream=stream)
        return out, lambda: pg.load().sk_norm_backward(ctypes.byref(a))
    return call


def test_backward_calls_of_several_threads():
    work = [[_block_backward(200, 300, 400), _block_backward(900, 700, 500)],
            [_block_backward(640, 1000, 260, grid_cap=7), _bf16_backward(512, 256, 1024)],
            [_bf16_backward(1024, 768, 512), _norm_backward(2000, 1000)],
            [_norm_backward(300, 4096), _block_backward(77, 130, 2000)]]
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    alone = []
    for calls in work:
        for call in calls:
            out, go = call(stream)
            assert go() == 0
            alone.append(out)
    torch.cuda.synchronize()
    pg.release_workspace()

    runs = [[call(stream) for _ in range(12) for call in calls] for calls in work]
    torch.cuda.synchronize()
    status = []
    start = threading.Barrier(len(runs))

    def loop(mine):
        start.wait()
        status.extend(go() for _, go in mine)

    threads = [threading.Thread(target=loop, args=(mine,)) for mine in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [0] * sum(map(len, runs))
    for i, mine in enumerate(runs):
        for k, (out, _) in enumerate(mine):
            want = alone[2 * i + k % 2]
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (i, k)


def test_backward_calls_give_the_interpreter_lock_up():
    """The native binding hands the call to whatever entry point it was given: here to the interpreter's own question
    whether this thread holds its lock, whose answer comes back as the call's status."""
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    x = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    w, r = x[0].clone(), torch.ones(16, device="cuda")
    qt, st = pg.quantize_fp8_block(x, transpose=True)
    bt, bst = pg.quantize_fp8_block(x, "tile", transpose=True)
    native = pg._native()
    dC = torch.zeros(16, 16, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    native.bind(held, held, held, held, held, torch._C._cuda_getCurrentRawStream)
    try:
        with pytest.raises(pg.SkError):      # (a call without scratch keeps it: the question is asked at all)
            pg.rms_norm(x, w)
        pg.gemm_fp8_block_backward(dC, qt, st, bt, bst)
        pg.rms_norm_backward(x, x, w, r)
    finally:
        pg._NATIVE = None
        pg._native()
    assert torch.equal(pg.rms_norm(x, w)[0], x)
