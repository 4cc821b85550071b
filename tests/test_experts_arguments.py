"""Arguments of the layer of experts' Python calls that are refused before any GPU work (no GPU is needed)."""

from __future__ import annotations

import pytest
import torch

import persistent_gemm_amd as pg


@pytest.mark.parametrize("bad", [2.5, 1.999, float("nan"), float("inf"), "x", "2"])
def test_sizes_are_whole_numbers(bad):
    """A fraction is refused, not cut off."""
    with pytest.raises((ValueError, OverflowError), match="k is|cannot convert|invalid literal"):
        pg.moe_route(torch.zeros(4, 8), bad)
    with pytest.raises((ValueError, OverflowError), match="group is|cannot convert|invalid literal"):
        pg.quantize_w4(torch.zeros(4, 128), bad)
    for call in (lambda: pg.moe_route(torch.zeros(4, 8), None), lambda: pg.quantize_w4(torch.zeros(4, 128), None)):
        with pytest.raises(TypeError):
            call()
    for whole in (2, 2.0):      # (no objection to the number itself)
        with pytest.raises(ValueError, match="expected a GPU"):
            pg.moe_route(torch.zeros(4, 8), whole)
    for whole in (64, 64.0):
        with pytest.raises(ValueError, match="expected a GPU"):
            pg.quantize_w4(torch.zeros(4, 128), whole)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its kernels would run there on tensors that are here."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    import persistent_gemm_amd.experts as experts

    class Stream:
        def __init__(self, index):
            self.device, self.cuda_stream = torch.device("cuda", index), 0

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with FakeTensorMode():
        x = torch.empty(4, 8, device="cuda:0")
        for stream in (Stream(1), Stream(7)):
            with pytest.raises(ValueError, match="stream is of cuda"):
                experts._on(x, "x", stream)
            for call in (lambda: pg.moe_route(x, 2, stream=stream), lambda: pg.moe_combine(x, x, stream=stream),
                         lambda: pg.quantize_w4(x, 32, stream=stream), lambda: pg.gemm_grouped(x, x[None], x, stream=stream)):
                with pytest.raises(ValueError, match="stream is of cuda"):
                    call()
        experts._on(x, "x", Stream(0))
