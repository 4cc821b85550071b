"""Limits and alignments that the header gives for the calls of a layer of experts: the least that each refuses (no GPU: the checks
come before any device work)."""

from __future__ import annotations

import pytest

from test_abi_experts import ALIGN, ARG, COMBINE, COMBINE_GRAD, DEQUANT, GROUPED, GROUPED_GRAD, P, QUANT, ROUTE, ROUTE_GRAD, W4, _status

ROWS = (1 << 31) - (1 << 20)


@pytest.mark.parametrize("name,base,kw,status", [
    ("sk_dequantize_w4", DEQUANT, dict(out=P[2] + 8), ALIGN), ("sk_dequantize_w4", DEQUANT, dict(scale=P[1] + 1), ALIGN),
    ("sk_moe_combine_backward", COMBINE_GRAD, dict(dy=P[5] + 8), ALIGN),
    ("sk_moe_combine_backward", COMBINE_GRAD, dict(dy=P[5] + 8, offsets=None), ALIGN),
    ("sk_gemm_grouped_backward", GROUPED_GRAD, dict(A=P[1] + 8), ALIGN), ("sk_gemm_grouped_backward", GROUPED_GRAD, dict(B=P[2] + 8), ALIGN),
    ("sk_gemm_grouped_backward", GROUPED_GRAD, dict(N=(1 << 21) + 8), ARG), ("sk_gemm_grouped_backward", GROUPED_GRAD, dict(K=(1 << 21) + 8), ARG),
    ("sk_gemm_grouped_backward", GROUPED_GRAD, dict(R=ROWS), ARG), ("sk_gemm_grouped", GROUPED, dict(R=ROWS), ARG),
    ("sk_moe_route", ROUTE, dict(T=ROWS, k=1), ARG), ("sk_moe_route_backward", ROUTE_GRAD, dict(E=1025), ARG),
    ("sk_moe_route_backward", ROUTE_GRAD, dict(E=64, k=33), ARG), ("sk_moe_combine", COMBINE, dict(R=ROWS + 1), ARG),
    ("sk_moe_combine_backward", COMBINE_GRAD, dict(k=33), ARG), ("sk_moe_combine_backward", COMBINE_GRAD, dict(D=(1 << 22) + 1), ARG),
    ("sk_quantize_w4", QUANT, dict(N=(1 << 22) + 1), ARG), ("sk_quantize_w4", QUANT, dict(K=(1 << 21) + 64), ARG),
    ("sk_dequantize_w4", DEQUANT, dict(E=1025), ARG), ("sk_dequantize_w4", DEQUANT, dict(N=0), ARG),
    ("sk_gemm_w4", W4, dict(N=(1 << 22) + 1), ARG), ("sk_gemm_w4", W4, dict(K=(1 << 21) + 64), ARG), ("sk_gemm_w4", W4, dict(T=0), ARG),
    ("sk_gemm_w4", W4, dict(M=ROWS), ARG),
])
def test_refuses(name, base, kw, status):
    assert _status(name, base, kw) == status
