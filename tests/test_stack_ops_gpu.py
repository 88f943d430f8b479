"""A decoder's linear parts as one stack: norms, 8-bit activations, activations,
multipliers and residuals around the layers (spear_w4ec_stack_set_op).  Every op's
output is checked against float64 fed the stack's own buffers."""
from __future__ import annotations

import pytest
import torch

from operator_refs import LayerRef, assert_bf16, assert_layer, norm_ref, norm_rel

pytestmark = pytest.mark.gpu

H, I = 256, 648          # hidden and inner width
EPS = 1e-5
# (in, out); 0 = x, 1 = y.  q reads norm(x); o adds x; gate, up read norm(o's output);
# down adds o's output
OPS = [("q", 0, 2), ("o", 2, 3), ("gate", 3, 4), ("up", 3, 5), ("down", 5, 1)]
SHAPES = {"q": (H, H), "o": (H, H), "gate": (H, I), "up": (H, I), "down": (I, H)}


class Block:
    def __init__(self, max_M, q8, r=16):
        from w4_gemm_error_b200.spear import W4ECStack
        self.q8 = q8
        self.lays = {n: LayerRef(*SHAPES[n], r if n != "o" else 0, seed=i) for i, n in enumerate(SHAPES)}
        self.lins = {n: lay.make(max_M) for n, lay in self.lays.items()}
        lay = self.lays["q"]
        self.w1 = (1 + 0.1 * lay.normal(H)).bfloat16()
        self.w2 = (1 + 0.1 * lay.normal(H)).bfloat16()
        self.bias = lay.normal(H).bfloat16()
        self.stack = W4ECStack([(self.lins[n], i, o, 1) for n, i, o in OPS], max_M)
        self.stack.set_op(0, norm=self.w1, eps=EPS, q8=q8, bias=self.bias)
        self.stack.set_op(1, residual=0, q8=q8)
        self.stack.set_op(2, norm=self.w2, eps=EPS, q8=q8, act="silu")
        self.stack.set_op(3, norm=self.w2, eps=EPS, q8=q8, mul=4)
        self.stack.set_op(4, residual=3, q8=q8)

    def activations(self, src, w=None):
        """What a layer reads, as the library makes it, in float64."""
        from w4_gemm_error_b200.spear import quantize_q8, rmsnorm
        if self.q8:
            q, s = quantize_q8(src) if w is None else rmsnorm(src, w, EPS, bf16=False, q8=True)[1:3]
            return q.double() * s.double()[:, None]
        if w is None:
            return src.double()
        y = rmsnorm(src, w, EPS)[0]
        assert_bf16(y, norm_ref(src, w, EPS)[1], norm_rel(H), "norm")
        return y.double()

    def check(self, x, y, ec=True):
        M = x.shape[0]
        b = {i: self.stack.buffer(i, M) for i in (2, 3, 4, 5)}
        L = self.lays
        assert_layer(b[2], L["q"], self.activations(x, self.w1), "q", ec=ec, bias=self.bias)
        assert_layer(b[3], L["o"], self.activations(b[2]), "o", ec=ec, residual=x)
        n2 = self.activations(b[3], self.w2)
        assert_layer(b[4], L["gate"], n2, "gate", ec=ec, act="silu")
        assert_layer(b[5], L["up"], n2, "up", ec=ec, mul=b[4])
        assert_layer(y, L["down"], self.activations(b[5]), "down", ec=ec, residual=b[3])
        assert all(lin.status() == 0 for lin in self.lins.values())


@pytest.mark.parametrize("q8", [False, True])
def test_block_at_several_batch_sizes(q8):
    from w4_gemm_error_b200.spear import SPEAR_EC_OFF
    blk = Block(300, q8)
    for M in (1, 9, 16, 17, 40, 130, 300, 1):
        x = (blk.lays["q"].normal(M, H) * 2).bfloat16()
        was = x.clone()
        y = blk.stack(x)
        blk.check(x, y)
        y = blk.stack(x, flags=SPEAR_EC_OFF)
        blk.check(x, y, ec=False)
        assert torch.equal(x, was)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_captured_block(q8, M):
    blk = Block(M, q8)
    x = blk.lays["q"].normal(M, H).bfloat16()
    y = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    blk.stack(x, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blk.stack(x, out=y)
    for _ in range(3):
        x.copy_(blk.lays["q"].normal(M, H))
        g.replay()
        blk.check(x, y)


def test_host_buffers_and_resetting_ops():
    from w4_gemm_error_b200 import spear
    blk = Block(8, True)
    x = blk.lays["q"].normal(4, H).bfloat16()
    xh, yh = x.cpu().pin_memory(), torch.empty(4, H, dtype=torch.bfloat16).pin_memory()
    blk.stack.forward_host(xh, yh)
    blk.check(x, yh.cuda())
    with pytest.raises(spear.SpearError) as e:
        blk.stack(x, flags=spear.SPEAR_STACK_PERSISTENT)
    assert e.value.status == spear.SPEAR_ERR_UNSUPPORTED
    for i in range(5):
        blk.stack.set_op(i)
    bare = spear.W4ECStack([(blk.lins[n], i, o, 1) for n, i, o in OPS], 8)
    assert torch.equal(blk.stack(x), bare(x))
    y = blk.stack(x, flags=spear.SPEAR_STACK_PERSISTENT)
    assert torch.isfinite(y).all()


def test_a_buffer_written_again_is_normed_again():
    """Two ops norm one buffer with one weight; in between it is overwritten."""
    from w4_gemm_error_b200.spear import W4ECStack
    lay = LayerRef(H, H, 8, seed=31)
    lin = lay.make(8)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    st = W4ECStack([(lin, 0, 2, 1), (lin, 2, 3, 1), (lin, 3, 2, 1), (lin, 2, 1, 1)], 8)
    for i in (1, 3):
        st.set_op(i, norm=w, eps=EPS)
    x = lay.normal(3, H).bfloat16()
    y = st(x)
    from w4_gemm_error_b200.spear import rmsnorm
    assert_layer(y, lay, rmsnorm(st.buffer(2, 3), w, EPS)[0].double(), "last")
    # in place: the op that overwrites the buffer it adds
    st.set_op(2, residual=2)
    b3 = st.buffer(3, 3)
    y = st(x)
    first = lin.forward(x)
    assert_layer(st.buffer(2, 3), lay, b3.double(), "in place", residual=first)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("M", [1, 30, 200])
def test_output_in_the_place_of_the_input(q8, M):
    """x is normed by the first op and added by the second, y written by the last."""
    blk = Block(M, q8)
    x = blk.lays["q"].normal(M, H).bfloat16()
    want, was = blk.stack(x), x.clone()
    assert blk.stack(x, out=x) is x
    assert torch.equal(x, want)
    blk.check(was, x)


def test_output_over_what_the_last_op_reads():
    from w4_gemm_error_b200 import spear
    lay = LayerRef(H, H, 8, seed=37)
    lin = lay.make(8)
    st = spear.W4ECStack([(lin, 0, 2, 1), (lin, 0, 1, 1)], 8)
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    flat = lay.normal(6 * H).bfloat16()
    x, shifted = flat[:4 * H].view(4, H), flat[8:8 + 4 * H].view(4, H)

    def refused(out):
        with pytest.raises(spear.SpearError) as e:
            st(x, out=out)
        assert e.value.status == spear.SPEAR_ERR_INVALID

    st.set_op(1, act="relu")                # the layer reads x itself
    refused(x)
    refused(shifted)
    st.set_op(1, residual=0, q8=True)       # x is quantised before, and added element by element
    refused(shifted)
    st.set_op(1, norm=w, bias=flat[2 * H:3 * H])
    refused(x)                              # the bias lies in y
    st.set_op(1, norm=w, residual=0)
    want = st(x)
    assert torch.equal(st(x, out=x), want)


def test_refusals():
    from w4_gemm_error_b200 import spear
    blk = Block(8, False)
    st = blk.stack
    for bad in (dict(mul=1), dict(mul=9), dict(residual=4), dict(residual=-2), dict(mul=2)):
        with pytest.raises(spear.SpearError) as e:     # (op 2 writes I columns; 4 is its own output, unwritten)
            st.set_op(2, **bad)
        assert e.value.status == spear.SPEAR_ERR_INVALID, bad
    with pytest.raises(spear.SpearError):
        st.set_op(2, norm=blk.w2, eps=float("nan"))
    for bad in (dict(norm=blk.w2[:8]), dict(bias=blk.bias), dict(act="tanh"), dict(norm=blk.w2.float())):
        with pytest.raises(ValueError):
            st.set_op(2, **bad)
    L = spear.lib()
    ext = spear.StackExt(None, 0.0, 0, None, 0, -1, -1)
    import ctypes
    assert L.spear_w4ec_stack_set_op(st.h, 5, ctypes.byref(ext)) == spear.SPEAR_ERR_INVALID
    assert L.spear_w4ec_stack_set_op(st.h, -1, ctypes.byref(ext)) == spear.SPEAR_ERR_INVALID
    assert L.spear_w4ec_stack_set_op(None, 0, ctypes.byref(ext)) == spear.SPEAR_ERR_INVALID
    bad = spear.StackExt(None, 0.0, 2, None, 0, -1, -1)
    assert L.spear_w4ec_stack_set_op(st.h, 0, ctypes.byref(bad)) == spear.SPEAR_ERR_INVALID
    bad = spear.StackExt(None, 0.0, 0, None, 7, -1, -1)
    assert L.spear_w4ec_stack_set_op(st.h, 0, ctypes.byref(bad)) == spear.SPEAR_ERR_INVALID
    x = blk.lays["q"].normal(4, H).bfloat16()
    blk.check(x, st(x))      # nothing of the refused calls stayed
