"""Stages that ordinary loads read and copies overwrite are given back with a proxy fence.

A copy (TMA) reaches shared memory by the async proxy; the release of an mbarrier arrival orders
ordinary accesses alone.  Each reader therefore issues fence.proxy.async between its last load of a
stage and the arrival that lets the next copy start.  Read from the sources, on the CPU; the GPU
test below checks values where the missing fence showed.
"""
from __future__ import annotations

import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4_gemm_error_b200", "csrc")
# kernels whose stages are read by ordinary loads and refilled by copies, with no store in
# between that depends on what was read
RINGS = {"decode.cu": 2, "decode_stream.cu": 1, "stack_decode.cu": 2}


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", sorted(RINGS))
def test_rings_are_released_behind_a_fence(name):
    text = source(name)
    assert len(re.findall(r"\brelease_stage\(", text)) == RINGS[name]
    for m in re.finditer(r"\bmbar_arrive\((?:smem_addr\(&)?(\w*empty\w*)", text):
        before = text[:m.start()]
        assert re.search(r"fence_proxy_async_smem\(\);\s*bar_consumers\(\);\s*if \(tid == 0\)\s*for \([^)]*\)\s*$", before), m.group(0)


def test_the_release_fences_before_the_warp_meets():
    text = source("async_utils.cuh")
    body = text[text.index("void release_stage("):]
    body = body[:body.index("\n}")]
    order = [body.index(s) for s in ("fence_proxy_async_smem()", "__syncwarp()", "mbar_arrive(")]
    assert order == sorted(order)


def test_a_warp_that_refills_its_own_slot_fences_first():
    text = source("decode_stream.cu")
    refill = text.index("if (lane == 0 && i + p.g_slots < n_units)")
    assert re.search(r"fence_proxy_async_smem\(\);\s*__syncwarp\(\);\s*$", text[:refill])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["forward", "ec off", "split", "epilogue", "q8"])
@pytest.mark.parametrize("M", [16, 24, 25, 32, 64])
@pytest.mark.parametrize("K,N,r", [(4096, 14336, 64), (14336, 4096, 64), (4096, 4096, 32)])
def test_decode_kernels_values(K, N, r, M, kind):
    from operator_refs import LayerRef, assert_layer
    from w4_gemm_error_b200.spear import SPEAR_EC_OFF, SPEAR_FORCE_DECODE, SPEAR_FORCE_FUSED, SPEAR_FORCE_SPLIT
    lay = LayerRef(K, N, r, seed=M)
    lin = lay.make(M)
    x = lay.normal(M, K).bfloat16()
    q, s = (40 * x.float()).clamp(-448, 448).to(torch.float8_e4m3fn), torch.ones(M, device="cuda")
    call = {"forward": lambda: lin.forward(x, flags=SPEAR_FORCE_DECODE | SPEAR_FORCE_FUSED),
            "ec off": lambda: lin.forward(x, flags=SPEAR_FORCE_DECODE | SPEAR_EC_OFF),
            "split": lambda: lin.forward(x, flags=SPEAR_FORCE_DECODE | SPEAR_FORCE_SPLIT),
            "epilogue": lambda: lin.forward_ep(x, act="relu", flags=SPEAR_FORCE_DECODE),
            "q8": lambda: lin.forward_q8(q, s, act="relu", flags=SPEAR_FORCE_DECODE)}[kind]
    got = [call() for _ in range(12)]
    x64 = q.double() if kind == "q8" else x.double()
    Y, E = lay.product(x64, kind != "ec off")
    if kind == "split":      # the product is rounded to bf16 before the correction is added
        base, _ = lay.product(x64, False)
        E = E + base.abs() * 2.0 ** -8
    if kind in ("epilogue", "q8"):
        Y = Y.clamp(min=0)
    tol = E + (Y.abs() + E) * (2.0 ** -8 + 2.0 ** -22) + 2.0 ** -133
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for y in got:
        bad += (~((y.double() - Y).abs() <= tol)).sum()
        bad += (y != got[0]).sum()
    assert bad.item() == 0
    if kind in ("epilogue", "q8"):
        assert_layer(got[0], lay, x64, kind, act="relu")
    assert lin.status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("K,N,r", [(4096, 14336, 64), (14336, 4096, 64), (4096, 4096, 32)])
def test_cluster_split_decode_values(K, N, r, M, monkeypatch):
    """The decode kernel with K split over a cluster (SPEAR_DECODE_STREAM)."""
    from operator_refs import LayerRef, assert_layer
    from w4_gemm_error_b200.spear import SPEAR_FORCE_DECODE, SPEAR_FORCE_FUSED
    monkeypatch.setenv("SPEAR_DECODE_STREAM", "1")
    lay = LayerRef(K, N, r, seed=M)
    lin = lay.make(M)
    x = lay.normal(M, K).bfloat16()
    got = [lin.forward(x, flags=SPEAR_FORCE_DECODE | SPEAR_FORCE_FUSED) for _ in range(12)]
    assert_layer(got[0], lay, x.double(), "stream")
    assert all(torch.equal(y, got[0]) for y in got)
    assert lin.status() == 0
