"""How exactly the layer's sums are kept, apart from the outputs' rounding.

The call is given the negative of the rounded result as its residual, so that what it returns is
its fp32 error and the remainder, not the result.  The bound is on the root mean square over all
outputs, of terms that follow the accumulation's steps:

  a step (one MMA, 16 k at least) is off by at most two units of 2^-23 of the partial sum that it
  works on: one where its products are aligned, one where they are added (truncation allowed).
  By Minkowski's inequality the root mean square of all steps' errors together is at most the
  number of steps times 2 * 2^-23 times the root mean square of the partial sums; 16 more units
  cover the sum over up to 8 parts of K, the zero point, the scales and the residual.

The partial sums are those of the form that the kernels use: x (q - z), or for 8 bits, whose zero
point is apart, the larger ones of x q.
"""
from __future__ import annotations

import math

import pytest
import torch

from operator_refs import BF16_HALF, LayerRef, unpack_codes

UNIT = 2.0 ** -23


def rms(t):
    return t.double().pow(2).mean().sqrt().item()


def partial_rms(x, w, parts=16):
    """Root mean square of the partial sums of x w^T over 1/16, 2/16, ... of k (float64)."""
    K, total, squares = x.shape[1], 0, 0.0
    for i in range(parts):
        lo, hi = K * i // parts, K * (i + 1) // parts
        total = total + x[:, lo:hi] @ w[:, lo:hi].t()
        squares += rms(total) ** 2
    return math.sqrt(squares / parts)


def sum_units(K):
    return (2 * math.ceil(K / 16) + 16) * UNIT


def activations(gen_normal, M, K, kind, one_sign):
    v = gen_normal(M, K) * (40 if kind == "q8" else 1)
    if one_sign:
        v = v.abs()
    return v.clamp(-448, 448).to(torch.float8_e4m3fn) if kind == "q8" else v.bfloat16()


def tolerance(lay, x, kind):
    """Bound on the root mean square of the fp32 error of lay's outputs on x (float64)."""
    s = lay.s.double()[:, None]
    R = partial_rms(x, lay.W)
    if kind == "q8":
        q = unpack_codes(lay.codes, lay.K).double()
        R = max(R, partial_rms(x, q * s), rms(x.sum(1)) * rms(lay.z.double()[:, None] * s))
    T = sum_units(lay.K) * R
    if lay.r:
        A, B = lay.A.double(), lay.B.double()
        logit = x @ lay.wg.double() + lay.b_g
        g, u = torch.sigmoid(logit)[:, None], x @ A
        # both operands of the correction in tf32: half a unit of 2^-10 each
        T += 1.01 * 2.0 ** -10 * rms(g * (u.abs() @ B.abs()))
        T += sum_units(lay.K) * partial_rms(x, A.t()) * rms(B.abs().sum(0))
        T += sum_units(lay.K) * 0.25 * partial_rms(x, lay.wg.double()[None, :]) * rms(u @ B) + 16 * UNIT * rms(u @ B)
    return T


# (the row-CTA, split-K, tile and pair kernels)
SHAPES = [(4, 4096, 512), (8, 14336, 512), (3, 1032, 520), (40, 14336, 512), (40, 1032, 520), (130, 4096, 1000),
          (300, 14336, 4096), (2600, 1032, 512)]


@pytest.mark.gpu
@pytest.mark.parametrize("r", [0, 64])
@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_sums_are_kept_in_32_bits(M, K, N, kind, one_sign, r):
    """one_sign: activations after a ReLU, for which the zero point's two terms are many times
    their difference."""
    lay = LayerRef(K, N, r, seed=M + K, asym=not one_sign)
    lin = lay.make(M)
    xin = activations(lay.normal, M, K, kind, one_sign)
    x = xin.double()
    Y, _ = lay.product(x)
    near = Y.bfloat16()
    if kind == "q8":
        got = lin.forward_q8(xin, torch.ones(M, device="cuda"), residual=-near)
    else:
        got = lin.forward_ep(xin, residual=-near)
    left = Y - near.double()
    T = tolerance(lay, x, kind)
    err = rms(got.double() - left)
    assert err <= T + BF16_HALF * (rms(left) + T), (err, T, rms(left), rms(Y))
    assert lin.status() == 0


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("K", [1032, 4096, 14336])
def test_the_bound_tells_32_bits_from_fewer(K, one_sign):
    """Sums in fp32 pass; planted: sums kept in 12 to 14 bits do not.  (On the CPU, steps of 16 k.)"""
    g = torch.Generator().manual_seed(K)
    M, N = 4, 96
    x = torch.randn(M, K, generator=g).bfloat16().double()
    x = x.abs() if one_sign else x
    w = (torch.randint(0, 16, (N, K), generator=g) - 8).double() * 2.0 ** -8
    exact = x @ w.t()
    T = sum_units(K) * partial_rms(x, w)

    def summed(bits):
        acc = torch.zeros(M, N, dtype=torch.float64)
        for k in range(0, K, 16):
            acc = acc + x[:, k:k + 16] @ w[:, k:k + 16].t()
            m, e = torch.frexp(acc)
            acc = torch.ldexp(torch.round(m * 2.0 ** bits) * 2.0 ** -bits, e)
        return rms(acc - exact)

    assert summed(24) <= T
    for bits in (12, 13, 14):
        assert summed(bits) > T, bits
