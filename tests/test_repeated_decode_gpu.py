"""Decode kernels replayed many times: a stage of their rings that was given back before its
loads were performed would show as outputs that differ from the first call's."""
from __future__ import annotations

import pytest
import torch

from operator_refs import LayerRef

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["forward", "epilogue", "q8"])
@pytest.mark.parametrize("M", [1, 8, 16, 32])
@pytest.mark.parametrize("K,N,r", [(14336, 4096, 64), (14336, 1024, 128), (8192, 4096, 0), (4104, 1000, 16)])
def test_every_form_of_the_decode_kernels_repeats(K, N, r, M, kind):
    from w4_gemm_error_b200.spear import SPEAR_FORCE_DECODE, SPEAR_FORCE_FUSED
    lays = [LayerRef(K, N, r, seed=i) for i in range(2)]
    lins = [lay.make(M) for lay in lays]
    x = [lay.normal(M, K).bfloat16() for lay in lays]
    q = [(40 * v.float()).clamp(-448, 448).to(torch.float8_e4m3fn) for v in x]
    s = torch.ones(M, device="cuda")

    def call(i):
        if kind == "forward":
            return lins[i].forward(x[i], flags=SPEAR_FORCE_DECODE | SPEAR_FORCE_FUSED)
        if kind == "epilogue":
            return lins[i].forward_ep(x[i], act="relu", flags=SPEAR_FORCE_DECODE)
        return lins[i].forward_q8(q[i], s, act="relu", flags=SPEAR_FORCE_DECODE)

    first = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(i % 2) for i in range(20)]
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(20):
        graph.replay()
        for i, y in enumerate(got):
            bad += (y != first[i % 2]).sum()
    assert bad.item() == 0
    assert all(lin.status() == 0 for lin in lins)
