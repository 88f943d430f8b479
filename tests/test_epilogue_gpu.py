"""The W4 + EC forward with bias, activation, multiplier and residual, on bf16 and
on 8-bit activations, against float64."""
from __future__ import annotations

import pytest
import torch

from operator_refs import LayerRef, assert_layer

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def bf16_x(lay, M):
    x = lay.normal(M, lay.K)
    x[:, ::61] *= 10
    return x.bfloat16()


def q8_x(lay, M):
    """Codes of any value and scales of several magnitudes."""
    q = (lay.normal(M, lay.K) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.exp(lay.normal(M)) * 0.02
    return q, s


def operands(lay, M, bias, mul, residual):
    return dict(bias=lay.normal(lay.N).bfloat16() if bias else None,
                mul=lay.normal(M, lay.N).bfloat16() if mul else None,
                residual=(3 * lay.normal(M, lay.N)).bfloat16() if residual else None)


def run(lin, lay, M, kind, flags=0, **ep):
    """(output, x in float64)"""
    if kind == "bf16":
        x = bf16_x(lay, M)
        return lin.forward_ep(x, flags=flags, **ep), x.double()
    q, s = q8_x(lay, M)
    return lin.forward_q8(q, s, flags=flags, **ep), q.double() * s.double()[:, None]


# M: around the kernels' token tiles; K, N: off their tiles, with and without the
# row-CTA kernel (K a multiple of 64); ranks with and without padding
CASES = [(1, 64, 128, 8), (2, 4096, 4096, 32), (7, 8, 8, 0), (8, 72, 136, 3), (9, 256, 1000, 16), (16, 4096, 512, 64),
         (17, 1032, 2744, 8), (31, 2056, 264, 128), (32, 512, 640, 15), (33, 520, 136, 24), (64, 4096, 1024, 64),
         (65, 264, 392, 0), (100, 1032, 520, 100), (128, 2048, 768, 32), (129, 272, 136, 31), (257, 1040, 1000, 64),
         (300, 4104, 264, 128), (513, 528, 3000, 16),
         # enough tiles for the kernel on pairs of CTAs, with a second CTA that has no channels,
         # ragged tokens, channels and K, and very few channels
         (4100, 1032, 520, 24), (2600, 264, 1000, 0), (9500, 72, 136, 8), (10000, 136, 8, 3), (1100, 4096, 2744, 128),
         # the same kernel with fewer tokens than one tile of it
         (40, 520, 9480, 24), (100, 264, 9608, 8), (128, 136, 19000, 0), (65, 72, 19200, 128)]


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M,K,N,r", CASES)
def test_against_float64(kind, M, K, N, r):
    i = CASES.index((M, K, N, r))
    lay = LayerRef(K, N, r, seed=i, asym=i % 2 == 0, zero_rows=i % 5 == 3)
    lin = lay.make(M)
    for k, act in enumerate(ACTS):
        ep = dict(act=act, **operands(lay, M, bias=(i + k) % 2 == 0, mul=(i + k) % 3 == 0, residual=(i + k) % 3 == 1))
        y, x = run(lin, lay, M, kind, **ep)
        assert_layer(y, lay, x, (kind, act), **ep)
    assert lin.status() == 0


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("path", ["decode", "tcgen05"])
@pytest.mark.parametrize("M", [1, 8, 33, 60, 100, 260])
@pytest.mark.parametrize("K,N,r", [(1032, 520, 40), (4096, 256, 32), (520, 136, 0)])
def test_either_kernel_family_at_any_size(kind, path, M, K, N, r):
    from w4_gemm_error_b200.spear import SPEAR_FORCE_DECODE, SPEAR_FORCE_TC
    lay = LayerRef(K, N, r, seed=M)
    lin = lay.make(M)
    ep = dict(act="silu", **operands(lay, M, True, False, True))
    y, x = run(lin, lay, M, kind, flags=SPEAR_FORCE_DECODE if path == "decode" else SPEAR_FORCE_TC, **ep)
    assert_layer(y, lay, x, (kind, path), **ep)
    assert lin.status() == 0


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M", [1, 5, 24, 70, 300, 4000])
def test_every_term_and_the_ec_off(kind, M):
    from w4_gemm_error_b200.spear import SPEAR_EC_OFF
    lay = LayerRef(1024, 520, 20, seed=3)
    lin = lay.make(M)
    ep = dict(act="silu", **operands(lay, M, True, True, True))
    y, x = run(lin, lay, M, kind, **ep)
    assert_layer(y, lay, x, "all", **ep)
    y, x = run(lin, lay, M, kind, flags=SPEAR_EC_OFF, **ep)
    assert_layer(y, lay, x, "ec off", ec=False, **ep)
    assert lin.status() == 0


@pytest.mark.parametrize("M", [1, 16, 20, 33, 64, 300])
@pytest.mark.parametrize("K,N,r", [(4096, 512, 32), (1032, 264, 8), (512, 640, 0)])
def test_no_epilogue_is_the_forward_bit_for_bit(M, K, N, r):
    from w4_gemm_error_b200.spear import SPEAR_FORCE_FUSED
    lay = LayerRef(K, N, r, seed=5)
    lin = lay.make(M)
    x = bf16_x(lay, M)
    assert torch.equal(lin.forward_ep(x), lin.forward(x, flags=SPEAR_FORCE_FUSED))


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M", [1, 9, 31, 64, 200, 5000])
def test_in_place_residual_and_multiplier(kind, M):
    lay = LayerRef(2048, 392, 16, seed=7)
    lin = lay.make(M)
    for names in (("residual",), ("mul",), ("residual", "mul")):
        buf = lay.normal(M, lay.N).bfloat16()
        was = buf.clone()
        y, x = run(lin, lay, M, kind, act="gelu", out=buf, **{n: buf for n in names})
        assert y is buf
        assert_layer(y, lay, x, names, act="gelu", **{n: was for n in names})


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M", [1, 12, 20, 40, 140, 4899])
def test_rows_past_the_last_are_left_alone(kind, M):
    lay = LayerRef(512, 264, 8, seed=9)
    lin = lay.make(M)
    big = torch.full((M + 8, lay.N), 5, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros(M, lay.N, dtype=torch.bfloat16, device="cuda")
    run(lin, lay, M, kind, out=big[:M], residual=res)
    assert (big[M:] == 5).all()


@pytest.mark.parametrize("M", [1, 8, 16, 30, 33, 100, 300, 4997])
def test_a_bad_token_stays_in_its_row(M):
    """NaN codes, NaN and infinite scales, infinite residuals reach only their own tokens."""
    lay = LayerRef(1024, 264, 16, seed=11)
    lin = lay.make(M)
    q, s = q8_x(lay, M)
    x = q.double() * s.double()[:, None]
    t = M // 2
    good = torch.arange(M, device="cuda") != t
    bad = q.view(torch.uint8).clone()
    bad[t, 77] = 0x7F
    y = lin.forward_q8(bad.view(torch.float8_e4m3fn), s)
    assert torch.isnan(y[t]).all()
    if M > 1:
        assert_layer(y[good], lay, x[good], "beside a NaN code")
    for v in (float("nan"), float("inf")):
        s2 = s.clone()
        s2[t] = v
        y = lin.forward_q8(q, s2)
        assert not torch.isfinite(y[t]).any()
        if M > 1:
            assert_layer(y[good], lay, x[good], "beside a bad scale")
    res = torch.zeros(M, lay.N, dtype=torch.bfloat16, device="cuda")
    res[t, 3] = float("inf")
    y = lin.forward_q8(q, s, residual=res)
    assert y[t, 3] == float("inf") and torch.isfinite(y[t, 4:]).all()


@pytest.mark.parametrize("M", [1, 20, 64, 300, 5000])
def test_extreme_codes(M):
    """All codes at the largest magnitude, all at the smallest, zeros, one sign, every zero point."""
    lay = LayerRef(2048, 264, 8, seed=13)
    lin = lay.make(M)
    s = torch.full((M,), 0.01, device="cuda")
    for v in (448.0, -448.0, 2.0 ** -9, -(2.0 ** -9), 0.0, 0.875 * 2.0 ** -6):
        q = torch.full((M, lay.K), v, device="cuda").to(torch.float8_e4m3fn)
        assert_layer(lin.forward_q8(q, s), lay, q.double() * s.double()[:, None], v)


def test_offsets_past_32_bits():
    """Outputs and operands whose element offsets leave 32 bits."""
    lay = LayerRef(64, 14336, 0, seed=15)
    M = 150016
    lin = lay.make(M)
    res = torch.zeros(M, lay.N, dtype=torch.bfloat16, device="cuda")
    tail = lay.normal(5, lay.N).bfloat16()
    res[-5:] = tail
    x = torch.zeros(M, lay.K, dtype=torch.bfloat16, device="cuda")
    x[-5:] = lay.normal(5, lay.K).bfloat16()
    y = lin.forward_ep(x, residual=res, out=res)
    assert_layer(y[-5:], lay, x[-5:].double(), "bf16", residual=tail)
    assert (y[1234] == 0).all()
    q = torch.zeros(M, lay.K, dtype=torch.float8_e4m3fn, device="cuda")
    q[-5:] = (lay.normal(5, lay.K) * 20).to(torch.float8_e4m3fn)
    s = torch.ones(M, device="cuda") * 0.1
    y.zero_()
    y[-5:] = tail
    y = lin.forward_q8(q, s, residual=y, out=y)
    assert_layer(y[-5:], lay, q[-5:].double() * s[-5:].double()[:, None], "q8", residual=tail)
    assert (y[1234] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M", [1, 24, 64, 300, 5000])
def test_captured_calls_on_two_handles(kind, M):
    """Two captured forwards of two handles, replayed with new data, in turn."""
    lays = [LayerRef(1032, 264, 8, seed=17), LayerRef(1024, 520, 32, seed=18)]
    lins = [lay.make(M) for lay in lays]
    ins, graphs = [], []
    for lay, lin in zip(lays, lins):
        a = [bf16_x(lay, M)] if kind == "bf16" else list(q8_x(lay, M))
        res, out = lay.normal(M, lay.N).bfloat16(), torch.empty(M, lay.N, dtype=torch.bfloat16, device="cuda")
        f = lin.forward_ep if kind == "bf16" else lin.forward_q8
        f(*a, act="silu", residual=res, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(*a, act="silu", residual=res, out=out)
        ins.append((a, res, out))
        graphs.append(g)
    for _ in range(2):
        for lay, (a, res, out) in zip(lays, ins):
            new = [bf16_x(lay, M)] if kind == "bf16" else list(q8_x(lay, M))
            for t, n in zip(a, new):
                t.copy_(n)
            res.copy_(lay.normal(M, lay.N))
        for g in graphs:
            g.replay()
        for lay, (a, res, out) in zip(lays, ins):
            x = a[0].double() if kind == "bf16" else a[0].double() * a[1].double()[:, None]
            assert_layer(out, lay, x, "replay", act="silu", residual=res)
    assert all(lin.status() == 0 for lin in lins)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_calls_of_many_sizes_back_to_back(kind):
    """One handle, batch sizes that take different kernels in turn, nothing waited for between."""
    lay = LayerRef(1024, 1024, 32, seed=19)
    lin = lay.make(512)
    sizes = [1, 300, 16, 64, 2, 33, 512, 17, 128, 8]
    todo = []
    for M in sizes:
        ep = dict(act="silu", **operands(lay, M, True, False, True))
        y, x = run(lin, lay, M, kind, **ep)
        todo.append((y, x, ep))
    for M, (y, x, ep) in zip(sizes, todo):
        assert_layer(y, lay, x, M, **ep)
    assert lin.status() == 0


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("M,K,N,r", [(64, 14336, 4096, 64), (64, 8192, 4096, 0), (33, 14336, 1024, 128),
                                     (128, 4096, 4096, 32), (100, 2048, 14336, 16), (20, 4096, 4096, 128),
                                     (300, 4096, 1000, 64), (700, 4096, 6144, 64), (16, 14336, 4096, 64),
                                     (8, 14336, 4096, 64), (1, 4096, 14336, 64), (8, 4096, 4096, 32)])
def test_many_calls_agree(kind, M, K, N, r):
    """Calls of three layers in turn, nothing waited for between, all giving the same bits
    and the right values: an operand overwritten while it is still read shows here."""
    from w4_gemm_error_b200.spear import SPEAR_EC_OFF
    lays = [LayerRef(K, N, r, seed=i, asym=i == 1) for i in range(3)]
    lins = [lay.make(M) for lay in lays]
    args = [(bf16_x(lay, M),) if kind == "bf16" else q8_x(lay, M) for lay in lays]
    x = [a[0].double() if kind == "bf16" else a[0].double() * a[1].double()[:, None] for a in args]

    def call(i, flags=0):
        f = lins[i].forward_ep if kind == "bf16" else lins[i].forward_q8
        return f(*args[i], act="relu", flags=flags)

    first = [call(i) for i in range(3)]
    for i in range(3):
        assert_layer(first[i], lays[i], x[i], "first", act="relu")
    off = [call(i, SPEAR_EC_OFF) for i in range(3)]
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for n in range(60):
        i = n % 3
        bad += (call(i) != first[i]).sum()
        if n % 4 == 0:
            bad += (call(i, SPEAR_EC_OFF) != off[i]).sum()
    for n in range(30):
        got = [call(i) for i in range(3)]    # back to back
        for i in range(3):
            bad += (got[i] != first[i]).sum()
    assert bad.item() == 0
    assert all(lin.status() == 0 for lin in lins)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_two_handles_on_two_streams(kind):
    """Calls of all sizes of two layers, each on its own stream, at once."""
    lays = [LayerRef(1032, 520, 24, seed=41), LayerRef(1024, 1000, 40, seed=42)]
    lins = [lay.make(4200) for lay in lays]
    streams = [torch.cuda.Stream() for _ in lays]
    sizes = [4200, 1, 300, 16, 64, 12, 33, 200]
    args = [[(bf16_x(lay, M),) if kind == "bf16" else q8_x(lay, M) for M in sizes] for lay in lays]
    f = [lin.forward_ep if kind == "bf16" else lin.forward_q8 for lin in lins]
    want = [[f[i](*a, act="relu") for a in args[i]] for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for k in range(len(sizes)):
            for i in range(2):
                got[i].append((k, f[i](*args[i][k], act="relu", stream=streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for k, y in got[i]:
            assert torch.equal(y, want[i][k]), (i, sizes[k])
    for i, lay in enumerate(lays):
        a = args[i][0]
        assert_layer(want[i][0], lay, a[0].double() if kind == "bf16" else a[0].double() * a[1].double()[:, None],
                     "values", act="relu")
    assert all(lin.status() == 0 for lin in lins)


@pytest.mark.parametrize("r", [0, 8])
@pytest.mark.parametrize("M", [1, 24, 300, 2600])
def test_operands_from_the_call_before(M, r):
    """Bias, multiplier and residual that the call right before on the stream writes."""
    a, b = LayerRef(14336, 1000, 0, seed=41), LayerRef(264, 1000, r, seed=42)
    la, lb = a.make(max(M, 1)), b.make(M)
    x = bf16_x(b, M)
    first = [bf16_x(a, 1) for _ in range(8)]
    rows = [bf16_x(a, M) for _ in range(2)]
    want = []
    for v in first:
        bias = la.forward_ep(v)[0].clone()
        torch.cuda.synchronize()
        want.append(lb.forward_ep(x, bias=bias))
        torch.cuda.synchronize()
    bias, got = torch.zeros(1, 1000, dtype=torch.bfloat16, device="cuda"), []
    torch.cuda.synchronize()
    for v in first:
        la.forward_ep(v, out=bias)
        got.append(lb.forward_ep(x, bias=bias[0]))
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    for name in ("mul", "residual"):
        want = []
        for v in rows:
            o = la.forward_ep(v).clone()
            torch.cuda.synchronize()
            want.append(lb.forward_ep(x, **{name: o}))
            torch.cuda.synchronize()
        buf, got = torch.zeros(M, 1000, dtype=torch.bfloat16, device="cuda"), []
        torch.cuda.synchronize()
        for v in rows:
            la.forward_ep(v, out=buf)
            got.append(lb.forward_ep(x, **{name: buf}))
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_results_repeat_bit_for_bit():
    lay = LayerRef(4096, 520, 64, seed=21)
    for M in (1, 16, 24, 64, 300):
        lin = lay.make(M)
        q, s = q8_x(lay, M)
        first = lin.forward_q8(q, s, act="gelu")
        assert all(torch.equal(lin.forward_q8(q, s, act="gelu"), first) for _ in range(5))


def test_a_tuned_split_placement_is_not_followed():
    """A table that chose the separate EC kernel still gives a fused epilogue."""
    lay = LayerRef(512, 264, 8, seed=23)
    lin = lay.make(64)
    x = bf16_x(lay, 40)
    y = torch.empty(40, lay.N, dtype=torch.bfloat16, device="cuda")
    lin.tune(x, y)
    import json
    tab = json.loads(lin.table_json())
    for b in tab["buckets"]:
        if b.get("choice"):
            b["choice"] = b["choice"].replace("fused", "split")
    lin.load_table(json.dumps(tab))
    res = lay.normal(40, lay.N).bfloat16()
    was = res.clone()
    y = lin.forward_ep(x, residual=res, out=res)
    assert_layer(y, lay, x.double(), "split table", residual=was)


def test_refusals():
    from w4_gemm_error_b200 import spear
    lay = LayerRef(256, 264, 8, seed=25)
    lin = lay.make(16)
    x, (q, s) = bf16_x(lay, 4), q8_x(lay, 4)
    wide = lay.normal(4, lay.N).bfloat16()
    for bad in (dict(act="swish"), dict(act=None), dict(bias=wide), dict(bias=wide[0].float()),
                dict(mul=wide[:3]), dict(residual=wide.cpu()), dict(out=wide.float()),
                dict(residual=torch.empty(4, 2 * lay.N, dtype=torch.bfloat16, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            lin.forward_ep(x, **bad)
        with pytest.raises(ValueError):
            lin.forward_q8(q, s, **bad)
    with pytest.raises(ValueError):
        lin.forward_q8(x, s)
    with pytest.raises(ValueError):
        lin.forward_q8(q, s[:3])
    with pytest.raises(ValueError):
        lin.forward_q8(q, s.double())
    with pytest.raises(ValueError):
        lin.forward_ep(x[:, :128])
    big = bf16_x(lay, 17)
    for call in (lambda **k: lin.forward_ep(big, **k), lambda **k: lin.forward_q8(*q8_x(lay, 17), **k)):
        with pytest.raises(spear.SpearError) as e:      # more tokens than the handle holds
            call()
        assert e.value.status == spear.SPEAR_ERR_INVALID
    for call in (lambda **k: lin.forward_ep(x, **k), lambda **k: lin.forward_q8(q, s, **k)):
        with pytest.raises(spear.SpearError) as e:
            call(flags=spear.SPEAR_FORCE_SPLIT)
        assert e.value.status == spear.SPEAR_ERR_UNSUPPORTED
        with pytest.raises(spear.SpearError) as e:
            call(flags=spear.SPEAR_FORCE_DECODE | spear.SPEAR_FORCE_TC)
        assert e.value.status == spear.SPEAR_ERR_INVALID
        buf = torch.zeros(5 * lay.N, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(spear.SpearError) as e:      # residual one row behind the output
            call(out=buf[lay.N:].view(4, lay.N), residual=buf[:4 * lay.N].view(4, lay.N))
        assert e.value.status == spear.SPEAR_ERR_INVALID
        with pytest.raises(spear.SpearError) as e:      # off 16 bytes
            call(bias=buf[1:1 + lay.N])
        assert e.value.status == spear.SPEAR_ERR_INVALID
    xy = torch.zeros(4 * lay.N, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(spear.SpearError):               # the output over the activations
        lin.forward_ep(xy[:4 * lay.K].view(4, lay.K), out=xy.view(4, lay.N))
    ep = spear.Epilogue(None, None, None, 9, 0)
    assert spear.lib().spear_w4ec_forward_ep(lin.h, x.data_ptr(), wide.data_ptr(), 4, ep, 0, None) == \
        spear.SPEAR_ERR_INVALID
    assert lin.forward_ep(x[:0]).shape == (0, lay.N)
    assert lin.forward_q8(q[:0], s[:0]).shape == (0, lay.N)
    assert lin.status() == 0


def test_an_input_on_another_device_is_refused():
    lay = LayerRef(256, 264, 8, seed=26)
    lin = lay.make(4)
    x, (q, s) = bf16_x(lay, 4), q8_x(lay, 4)
    lin.device = torch.device("cuda", x.get_device() + 1)
    with pytest.raises(ValueError):
        lin.forward_ep(x)
    with pytest.raises(ValueError):
        lin.forward_q8(q, s)
