"""8-bit layers without an Error Compensator on both sides of the rule between the tile and the
pair kernel, against float64."""
from __future__ import annotations

import pytest
import torch

from operator_refs import LayerRef, assert_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("M,K,N", [(64, 1024, 9600), (128, 512, 14336), (384, 2056, 4096), (321, 264, 3000),
                                   (513, 1032, 2744), (1300, 4096, 1024), (2500, 136, 512), (4096, 72, 520)])
def test_without_the_ec(M, K, N, off):
    """off: a layer with an EC that the call leaves out."""
    from w4_gemm_error_b200.spear import SPEAR_EC_OFF
    lay = LayerRef(K, N, 16 if off else 0, seed=M, asym=M % 2 == 0)
    lin = lay.make(M)
    q = (lay.normal(M, K) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.exp(lay.normal(M)) * 0.02
    bias, mul = lay.normal(N).bfloat16(), lay.normal(M, N).bfloat16()
    flags = SPEAR_EC_OFF if off else 0
    for ep in (dict(), dict(act="silu", bias=bias), dict(act="gelu", bias=bias, mul=mul, residual=mul)):
        y = lin.forward_q8(q, s, flags=flags, **ep)
        assert_layer(y, lay, q.double() * s.double()[:, None], (M, K, N), ec=False, **ep)
    assert lin.status() == 0
