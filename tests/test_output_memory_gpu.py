"""Outputs that a call makes itself belong to the stream that it runs on."""
from __future__ import annotations

import pytest
import torch

from operator_refs import LayerRef

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose memory t lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not torch's memory")


@pytest.mark.parametrize("as_handle", [False, True])
def test_new_outputs_are_the_given_streams(as_handle):
    from w4_gemm_error_b200.spear import W4ECStack, quantize_q8, rmsnorm
    lay = LayerRef(256, 264, 8, seed=1)
    lin = lay.make(8)
    x, w = lay.normal(8, 256).bfloat16(), lay.normal(256).bfloat16()
    res = x.clone()
    q, s = quantize_q8(x)
    st = W4ECStack([(lin, 0, 1, 1)], max_M=8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h = side.cuda_stream if as_handle else side
    calls = {
        "rmsnorm": lambda k: rmsnorm(x, w, 1e-6, res, q8=True, stream=k),
        "quantize_q8": lambda k: quantize_q8(x, stream=k),
        "forward": lambda k: [lin.forward(x, stream=k)],
        "forward_ep": lambda k: [lin.forward_ep(x, act="relu", stream=k)],
        "forward_q8": lambda k: [lin.forward_q8(q, s, stream=k)],
        "gate": lambda k: [lin.gate(x, stream=k)],
        "packed": lambda k: lin.packed(stream=k),
        "stack": lambda k: [st.forward(x, stream=k)],
    }
    for name, call in calls.items():
        torch.cuda.synchronize()
        got = call(h)
        torch.cuda.synchronize()
        assert [stream_of(t) for t in got] == [side.cuda_stream] * len(got), name
        here = call(None)
        assert [stream_of(t) for t in here] == [torch.cuda.current_stream().cuda_stream] * len(here), name
        torch.cuda.synchronize()
        for a, b in zip(got, here):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
