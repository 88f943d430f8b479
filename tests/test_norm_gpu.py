"""Row norm with residual and 8-bit output, and 8-bit quantisation, against float64."""
from __future__ import annotations

import pytest
import torch

from operator_refs import assert_bf16, assert_codes, norm_ref, norm_rel

pytestmark = pytest.mark.gpu

EPS = 1e-6


def rows(M, K, seed=0, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda") * std
    x[:, ::97] *= 20
    return x.bfloat16()


SHAPES = [(1, 8), (1, 4096), (3, 1), (2, 7), (5, 31), (4, 66), (37, 2050), (9, 2048), (2, 4104), (33, 1032),
          (3, 14336), (2, 16384), (2, 16390), (1, 32768), (2, 40000), (1, 33001), (300, 256), (1, 131072),
          # many rows, with one to four vectors a thread and one warp upwards
          (700, 8), (1500, 64), (999, 264), (1201, 1032), (2049, 2048), (650, 4104), (800, 10000), (601, 14336),
          (1200, 16384), (593, 2050),
          # many short rows: a warp each
          (2371, 1), (2400, 8), (2371, 50), (3001, 33), (2369, 127), (4000, 512), (2999, 1024), (2500, 254)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_of_both_outputs(M, K, residual):
    from w4_gemm_error_b200.spear import rmsnorm
    x, w = rows(M, K, 1), (1 + 0.1 * rows(1, K, 2)[0].float()).bfloat16()
    res = rows(M, K, 3) if residual else None
    y, q, s, h = rmsnorm(x, w, EPS, res, q8=True)
    href, v = norm_ref(x, w, EPS, res)
    if residual:
        assert torch.equal(h, href)
    else:
        assert h is None
    assert_bf16(y, v, norm_rel(K), "y")
    assert_codes(q, s, v, norm_rel(K), "q")


@pytest.mark.parametrize("M,K", SHAPES)
def test_quantisation(M, K):
    from w4_gemm_error_b200.spear import quantize_q8
    x = rows(M, K, 4, std=3.0)
    q, s = quantize_q8(x)
    assert_codes(q, s, x.double(), 0.0, "q")


def test_single_outputs_equal_the_joint_call():
    from w4_gemm_error_b200.spear import rmsnorm
    x, w, res = rows(19, 1032, 1), rows(1, 1032, 2)[0], rows(19, 1032, 3)
    y, q, s, h = rmsnorm(x, w, EPS, res, q8=True)
    y1, q1, s1, h1 = rmsnorm(x, w, EPS, res)
    assert q1 is None and s1 is None and torch.equal(y1, y) and torch.equal(h1, h)
    y2, q2, s2, _ = rmsnorm(x, w, EPS, res, bf16=False, q8=True)
    assert y2 is None and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("M,K", [(7, 1032), (7, 2050), (7, 40000), (900, 1032), (700, 4096)])
def test_outputs_in_the_place_of_inputs(M, K):
    from w4_gemm_error_b200.spear import rmsnorm
    x, w, res = rows(M, K, 1), rows(1, K, 2)[0], rows(M, K, 3)
    y, _, _, h = rmsnorm(x, w, EPS, res)
    for sum_in, y_in in (("res", None), ("x", None), ("res", "x"), ("x", "res"), (None, "x"), (None, "res")):
        t = {"x": x.clone(), "res": res.clone(), None: None}
        y2, _, _, h2 = rmsnorm(t["x"], w, EPS, t["res"], out=t[y_in], out_sum=t[sum_in])
        assert torch.equal(y2, y) and torch.equal(h2, h), (sum_in, y_in)
    t = x.clone()
    y3, _, _, _ = rmsnorm(t, w, EPS, out=t)
    assert torch.equal(y3, rmsnorm(x, w, EPS)[0])


@pytest.mark.parametrize("M,K", [(8, 256), (8, 1030), (8, 40000), (800, 256), (700, 4104)])
def test_zero_tiny_and_bad_rows(M, K):
    from w4_gemm_error_b200.spear import quantize_q8, rmsnorm
    x = rows(M, K, 1)
    x[1] = 0
    x[2] = 1e-36
    x[3] = 1e30
    x[4, 5] = float("inf")
    x[5, K - 1] = float("nan")
    x[6, 3] = float("-inf")
    good = [0, 1, 2, 3, 7]
    q, s = quantize_q8(x)
    assert_codes(q[good], s[good], x[good].double(), 0.0, "q")
    assert (q[1].float() == 0).all() and s[1] > 0
    v = q.float() * s[:, None]
    assert torch.isfinite(v[good]).all()
    for t in (4, 5, 6):
        assert not torch.isfinite(s[t]) or torch.isnan(v[t]).any()
    assert not torch.isfinite(s[4]) and torch.isnan(s[5]) and not torch.isfinite(s[6])
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    y, q, s, _ = rmsnorm(x, w, EPS, q8=True)
    mild = [0, 1, 2, 7]   # (the squares of row 3 leave fp32)
    assert_bf16(y[mild], norm_ref(x[mild], w, EPS)[1], norm_rel(K), "y")
    assert_codes(q[mild], s[mild], norm_ref(x[mild], w, EPS)[1], norm_rel(K), "q")
    assert torch.isnan(y[5]).all() and torch.isnan(s[5])


@pytest.mark.parametrize("M", [5, 777])
def test_rows_past_the_last_are_left_alone(M):
    from w4_gemm_error_b200.spear import rmsnorm
    K = 1032
    w = rows(1, K, 2)[0]
    big = {n: torch.full((M + 4, K), 7, dtype=torch.bfloat16, device="cuda") for n in ("y", "h")}
    q = torch.full((M + 4, K), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((M + 4,), 7.0, device="cuda")
    rmsnorm(rows(M, K, 1), w, EPS, rows(M, K, 3), q8=True, out=big["y"][:M], out_q=q[:M], out_s=s[:M],
            out_sum=big["h"][:M])
    assert (big["y"][M:] == 7).all() and (big["h"][M:] == 7).all() and (s[M:] == 7).all()
    assert (q.view(torch.uint8)[M:] == 7).all()


@pytest.mark.parametrize("M,K", [(2371, 512), (2374, 65)])
def test_short_rows_in_place_and_past_the_last(M, K):
    from w4_gemm_error_b200.spear import quantize_q8, rmsnorm
    x, w, res = rows(M, K, 1), rows(1, K, 2)[0], rows(M, K, 3)
    y, _, _, h = rmsnorm(x, w, EPS, res)
    buf = torch.full((M + 9, K), 7, dtype=torch.bfloat16, device="cuda")
    buf[:M] = x
    r = res.clone()
    rmsnorm(buf[:M], w, EPS, r, out=buf[:M], out_sum=r)
    assert torch.equal(buf[:M], y) and torch.equal(r, h) and (buf[M:] == 7).all()
    q = torch.full((M + 9, K), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((M + 9,), 7.0, device="cuda")
    quantize_q8(x, out_q=q[:M], out_s=s[:M])
    assert_codes(q[:M], s[:M], x.double(), 0.0, "q")
    assert (q.view(torch.uint8)[M:] == 7).all() and (s[M:] == 7).all()


def test_offsets_past_32_bits():
    from w4_gemm_error_b200.spear import quantize_q8
    M, K = 262160, 8200          # 2.15e9 elements
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rows(3, K, 1)
    q, s = quantize_q8(x)
    assert_codes(q[-3:], s[-3:], x[-3:].double(), 0.0, "q")
    assert (q[1000].float() == 0).all()


def test_a_captured_call_reads_what_its_buffers_hold_at_replay():
    from w4_gemm_error_b200.spear import rmsnorm
    K = 2048
    x, w, res = rows(6, K, 1), rows(1, K, 2)[0], rows(6, K, 3)
    out = [torch.empty_like(x), torch.empty(6, K, dtype=torch.float8_e4m3fn, device="cuda"),
           torch.empty(6, device="cuda"), torch.empty_like(x)]

    def call():
        rmsnorm(x, w, EPS, res, q8=True, out=out[0], out_q=out[1], out_s=out[2], out_sum=out[3])

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    x.copy_(rows(6, K, 11))
    res.copy_(rows(6, K, 13))
    g.replay()
    h, v = norm_ref(x, w, EPS, res)
    assert torch.equal(out[3], h)
    assert_bf16(out[0], v, norm_rel(K), "y")
    assert_codes(out[1], out[2], v, norm_rel(K), "q")


def test_calls_on_two_streams():
    from w4_gemm_error_b200.spear import quantize_q8
    xs = [rows(64, 4096, 20 + i) for i in range(2)]
    want = [quantize_q8(x) for x in xs]
    st = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[quantize_q8(x, stream=t) for _ in range(5)] for x, t in zip(xs, st)]
    torch.cuda.synchronize()
    for calls, (q, s) in zip(got, want):
        for q2, s2 in calls:
            assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


def test_refusals():
    from w4_gemm_error_b200 import spear
    x, w = rows(4, 64, 1), rows(1, 64, 2)[0]
    for bad in (dict(x=x.float()), dict(x=x[:, ::2]), dict(weight=w[:32]), dict(weight=w.cpu()), dict(bf16=False),
                dict(residual=x[:2]), dict(out_sum=x.clone()), dict(out_q=x), dict(out=x[:2])):
        a = dict(x=x, weight=w) | bad
        with pytest.raises(ValueError):
            spear.rmsnorm(a.pop("x"), a.pop("weight"), EPS, **a)
    with pytest.raises(ValueError):
        spear.quantize_q8(x[0])
    buf = torch.zeros(4 * 64 + 64, dtype=torch.bfloat16, device="cuda")
    a, b = buf[:256].view(4, 64), buf[64:].view(4, 64)      # overlap by three rows
    with pytest.raises(spear.SpearError) as e:
        spear.rmsnorm(a, w, EPS, out=b)
    assert e.value.status == spear.SPEAR_ERR_INVALID
    with pytest.raises(spear.SpearError):
        spear.rmsnorm(x, w, EPS, x.clone(), out=a, out_sum=a)   # one buffer for both outputs
    with pytest.raises(spear.SpearError):
        spear.rmsnorm(x, w, -1.0)
    with pytest.raises(spear.SpearError):
        spear.rmsnorm(x, w, float("nan"))
    with pytest.raises(spear.SpearError):                     # rows that start off 16 bytes
        spear.rmsnorm(buf[1:257].view(4, 64), w, EPS)
    q = buf.view(torch.float8_e4m3fn)[:256].view(4, 64)
    with pytest.raises(spear.SpearError):
        spear.quantize_q8(a, out_q=q)
    assert spear.rmsnorm(x[:0], w, EPS)[0].shape == (0, 64)
