"""The activations far out, where their values approach bf16's smallest, against float64."""
from __future__ import annotations

import pytest
import torch

from operator_refs import BF16_HALF, LayerRef, activate

pytestmark = pytest.mark.gpu


# (the row-CTA, split-K, tile and pair kernels)
@pytest.mark.parametrize("M,K", [(1, 64), (3, 72), (40, 72), (2600, 64)])
@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_tails(act, kind, M, K):
    """An input of zeros, so that the bias is the activation's argument.

    Relative: a tail falls like exp(-c) with c <= 97 (gelu: c = v^2 / 2), whose argument takes
    at most three roundings of 2^-24 and one of its half in the exponent's unit: below 97 * 6 *
    2^-24 < 2^-14, beside erfc's and exp2's own units.  Absolute: what is smaller than bf16's
    smallest value, 2^-133, may be that or 0."""
    N = 512
    lay = LayerRef(K, N, 0, seed=3)
    lin = lay.make(M)
    bias = torch.linspace(-112, 8, N, device="cuda").bfloat16()
    if act != "silu":
        bias = torch.linspace(-16, 8, N, device="cuda").bfloat16()
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    if kind == "bf16":
        y = lin.forward_ep(x, act=act, bias=bias)
    else:
        y = lin.forward_q8(x.to(torch.float8_e4m3fn), torch.ones(M, device="cuda"), act=act, bias=bias)
    want = activate(bias.double(), act).expand(M, N)
    err = (y.double() - want).abs()
    tol = want.abs() * (BF16_HALF + 2.0 ** -14) + 2.0 ** -133
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), bias[bad[0]].tolist()[:4], y[0][bad[0]].tolist()[:4])
    assert lin.status() == 0
