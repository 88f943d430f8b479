"""Argument checks of the norm, quantisation, epilogue and stack-op calls that need no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

INVALID = -1
PTR, ODD = 1 << 20, (1 << 20) + 2      # never dereferenced: every call is refused before a launch


@pytest.fixture(scope="module")
def spear():
    from w4_gemm_error_b200 import build
    build.build(quiet=True)
    from w4_gemm_error_b200 import spear
    return spear


def test_rmsnorm_refusals(spear):
    f = spear.lib().spear_w4ec_rmsnorm
    M, K = 4, 64
    n = 2 * M * K
    x, r, w, h, y, q, s = (PTR + i * 4 * n for i in range(7))
    bad = [
        (None, None, w, 1e-6, M, K, None, y, None, None), (x, None, None, 1e-6, M, K, None, y, None, None),
        (x, None, w, 1e-6, M, K, None, None, None, None), (x, None, w, 1e-6, M, K, None, y, q, None),
        (x, None, w, 1e-6, M, K, None, y, None, s), (x, r, w, 1e-6, M, K, None, y, None, None),
        (x, None, w, 1e-6, M, K, h, y, None, None), (x, None, w, -1.0, M, K, None, y, None, None),
        (x, None, w, float("nan"), M, K, None, y, None, None), (x, None, w, float("inf"), M, K, None, y, None, None),
        (x, None, w, 1e-6, -1, K, None, y, None, None), (x, None, w, 1e-6, M, 0, None, y, None, None),
        (x, None, w, 1e-6, M, 1 << 31, None, y, None, None), (x, None, w, 1e-6, 1 << 31, K, None, y, None, None),
        (ODD, None, w, 1e-6, M, K, None, y, None, None), (x, None, ODD, 1e-6, M, K, None, y, None, None),
        (x, None, w, 1e-6, M, K, None, y + 2, None, None), (x, None, w, 1e-6, M, K, None, None, q + 8, s),
        (x, None, w, 1e-6, M, K, None, None, q, s + 2),
        # overlaps other than an output in the place of an input
        (x, None, w, 1e-6, M, K, None, x + 16, None, None), (x, r, w, 1e-6, M, K, y, y, None, None),
        (x, None, w, 1e-6, M, K, None, y, y, s), (x, None, w, 1e-6, M, K, None, None, x, s),
        (x, None, w, 1e-6, M, K, None, w, None, None), (x, r, w, 1e-6, M, K, r + 16, y, None, None),
        (x, None, w, 1e-6, M, K, None, None, q, x), (x, None, w, 1e-6, M, K, None, None, q, q),
    ]
    for a in bad:
        assert f(*a, None) == INVALID, a
    assert f(x, None, w, 1e-6, 0, K, None, y, None, None, None) == 0


def test_quantize_refusals(spear):
    f = spear.lib().spear_w4ec_quantize_q8
    M, K = 4, 64
    x, q, s = PTR, PTR + 4096, PTR + 8192
    for a in ((None, M, K, q, s), (x, M, K, None, s), (x, M, K, q, None), (x, -1, K, q, s), (x, M, 0, q, s),
              (x + 2, M, K, q, s), (x, M, K, q + 4, s), (x, M, K, q, s + 1), (x, M, K, x, s), (x, M, K, q, x),
              (x, M, K, q, q + 16)):
        assert f(*a, None) == INVALID, a
    assert f(x, 0, K, q, s, None) == 0


def test_null_handles(spear):
    L = spear.lib()
    ep = spear.Epilogue(None, None, None, 0, 0)
    ext = spear.StackExt(None, 0.0, 0, None, 0, -1, -1)
    assert L.spear_w4ec_forward_ep(None, None, None, 1, ctypes.byref(ep), 0, None) == INVALID
    assert L.spear_w4ec_forward_q8(None, None, None, None, 1, None, 0, None) == INVALID
    assert L.spear_w4ec_stack_set_op(None, 0, ctypes.byref(ext)) == INVALID


def test_binding_refuses_host_tensors_and_other_types(spear):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: spear.rmsnorm(x, x[0]), lambda: spear.quantize_q8(x), lambda: spear.rmsnorm(None, None),
                 lambda: spear.quantize_q8([1.0])):
        with pytest.raises(ValueError):
            call()
