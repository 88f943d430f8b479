"""8-bit activations whose scales are near the ends of fp32: rows of bf16's largest values
quantise to scales of 2^119, and every finite scale is a caller's to give."""
from __future__ import annotations

import pytest
import torch

from operator_refs import LayerRef, assert_layer

pytestmark = pytest.mark.gpu

# (the row-CTA, split-K, tile and pair kernels; the last two with the prepass where r > 0)
SHAPES = [(1, 64, 264, 8), (3, 72, 264, 8), (20, 264, 264, 8), (20, 264, 264, 0), (60, 1032, 520, 24),
          (2600, 264, 1000, 0), (4100, 1032, 520, 24)]


@pytest.mark.parametrize("M,K,N,r", SHAPES)
@pytest.mark.parametrize("exponent", [119, 120, -100])
def test_finite_scales_give_finite_outputs(exponent, M, K, N, r):
    """|y| <= 2^exponent K 448 15 s |EC| is far from fp32's end only for few large codes: the codes
    are drawn from +-{0 .. 2}, so that |Y| stays below 2^120 2 1032 15 0.006 < 2^128.  Every third
    weight row has the scale 0 (weights 0)."""
    lay = LayerRef(K, N, r, seed=7, asym=True, zero_rows=True)
    lin = lay.make(M)
    q = lay.normal(M, K).clamp(-2, 2).to(torch.float8_e4m3fn)
    s = torch.full((M,), 2.0 ** exponent, device="cuda")
    y = lin.forward_q8(q, s)
    assert torch.isfinite(y).all()
    assert_layer(y, lay, q.double() * s.double()[:, None], exponent)
    assert lin.status() == 0


@pytest.mark.parametrize("M", [1, 20, 2600])
def test_rows_of_the_largest_values(M):
    """quantize_q8 of rows with bf16's largest value, through a layer."""
    from w4_gemm_error_b200.spear import quantize_q8
    lay = LayerRef(264, 1000, 0, seed=9)
    lin = lay.make(M)
    x = lay.normal(M, 264).bfloat16()
    x[:, 5] = torch.finfo(torch.bfloat16).max
    q, s = quantize_q8(x)
    assert (s >= 2.0 ** 119).all()
    y = lin.forward_q8(q, s)
    assert torch.isfinite(y).all()
    assert_layer(y, lay, q.double() * s.double()[:, None], "largest")
