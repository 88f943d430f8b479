"""Plain 64-bit references and derived tolerances of the operators around the
W4 + EC layer (row norm, 8-bit quantisation, forward with an epilogue)."""
from __future__ import annotations

import math

import torch

FLOOR = 2.0 ** -100
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2   # 2^-8
E4M3_HALF = torch.finfo(torch.float8_e4m3fn).eps / 2   # 2^-4
E4M3_SUB_HALF = 2.0 ** -10                        # half of the smallest e4m3 step


def norm_ref(x, w, eps, residual=None):
    """(h bf16, v float64): h is exact (one fp32 addition, one rounding)."""
    h = x if residual is None else (x.float() + residual.float()).bfloat16()
    d = h.double()
    v = d * w.double() / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    return h, v


def quant_ref(v):
    """(v in units of the row's scale, scale), both float64."""
    a = v.abs().amax(1, keepdim=True).clamp(min=FLOOR)
    return v * 448 / a, (a / 448).flatten()


# fp32 arithmetic of the norm: at most 32 squares a thread and 10 levels of a
# tree in the sum, then a square root, a reciprocal and three products: below
# 64 roundings of 2^-24, and for a row longer than the registers hold 32 + K / 8192
def norm_rel(K):
    return (64 + K / 8192) * 2.0 ** -24


def assert_bf16(got, want, rel, what):
    err = (got.double() - want).abs()
    tol = want.abs() * (BF16_HALF + 2 * rel) + 2.0 ** -133   # the last: bf16's subnormals
    bad = err > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), err[bad][0].item())


def assert_codes(q, s, v, rel, what):
    """q (e4m3) and s against v (float64): each code within half a step of v / s,
    the scale within its fp32 roundings."""
    t, sr = quant_ref(v)
    assert ((s.double() - sr).abs() <= sr * (rel + 4 * 2.0 ** -24)).all(), what
    err = (q.double() - t).abs()
    tol = torch.maximum(t.abs() * E4M3_HALF, torch.full_like(t, E4M3_SUB_HALF)) + t.abs() * (rel + 2.0 ** -20)
    bad = err > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


def activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    assert act == "none"
    return v


def unpack_codes(codes, K):
    sh = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    return ((codes.view(torch.int32).unsqueeze(2) >> sh) & 15).reshape(codes.shape[0], K)


class LayerRef:
    """A random packed layer on the GPU and its product in float64, with a bound
    on the fp32 rounding of the kernels' sums."""

    def __init__(self, K, N, r, seed=0, asym=True, zero_rows=False, device="cuda"):
        from w4_gemm_error_b200.spear import W4ECLinear
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.K, self.N, self.r = K, N, r

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device=device) * std

        q = torch.randint(0, 16, (N, K), generator=g, device=device, dtype=torch.int32)
        self.z = (torch.randint(0, 16, (N,), generator=g, device=device, dtype=torch.int32) if asym else
                  torch.full((N,), 8, device=device, dtype=torch.int32)).to(torch.uint8)
        self.s = (torch.rand(N, generator=g, device=device) + 0.5) * 0.004
        if zero_rows:
            self.s[:: 3] = 0
        codes = torch.zeros(N, K // 8, dtype=torch.int32, device=device)
        for i in range(8):
            codes |= q[:, i::8] << (4 * i)
        self.codes = codes
        self.W = (q.double() - self.z.double()[:, None]) * self.s.double()[:, None]
        self.A = self.B = self.wg = None
        self.b_g = -0.3
        if r:
            self.A = normal(K, r, std=0.02).bfloat16()
            self.B = normal(r, N, std=0.2).bfloat16()
            self.wg = normal(K, std=1 / math.sqrt(K)).bfloat16()
        self.gen, self.normal, self.device = g, normal, device
        self.make = lambda max_M: W4ECLinear(None, self.A, self.B, self.wg, self.b_g, max_M=max_M,
                                             packed=(self.codes, self.s, self.z))

    def product(self, x, ec=True):
        """(Y, bound on the kernels' error in Y) for x in float64.

        Every product is exact in fp32 (at most 8 + 5 significant bits), so the
        main sum is off by at most K roundings of 2^-24 of the sum of
        magnitudes; u, g and the correction likewise, and the tcgen05 kernels
        round the correction's two operands to tf32 (2^-11 each).  Sums of codes
        that keep the zero point apart are of magnitudes up to 15 / |q - z|
        times larger: the bound takes |q - z| as 15."""
        Y = x @ self.W.t()
        E = (self.K + 64) * 2.0 ** -24 * (x.abs().sum(1, keepdim=True) * (15 * self.s.double())[None, :])
        if self.r and ec:
            A, B, wg = self.A.double(), self.B.double(), self.wg.double()
            u, logit = x @ A, x @ wg + self.b_g
            ua, la = x.abs() @ A.abs(), x.abs() @ wg.abs()
            gate = torch.sigmoid(logit)
            Y = Y + gate[:, None] * (u @ B)
            rel = (self.K + self.r + 64) * 2.0 ** -24
            dgate = gate * (1 - gate) * (la + 1) * rel + 8 * 2.0 ** -24
            E = E + (rel * gate[:, None] * (ua @ B.abs()) + dgate[:, None] * (u.abs() @ B.abs())
                     + 2.0 ** -10 * 1.01 * gate[:, None] * (u.abs() @ B.abs()))
        return Y, E


def assert_layer(got, lay, x, what, ec=True, act="none", bias=None, mul=None, residual=None):
    """got (bf16) against act(Y + bias) * mul + residual.  No activation has a
    slope above 1.13; its fast exponential is off by less than 2^-16 relative."""
    Y, E = lay.product(x, ec)
    if bias is not None:
        Y = Y + bias.double()
    v = activate(Y, act)
    E = 1.13 * E + 2.0 ** -16 * v.abs() + 2.0 ** -24 * Y.abs()
    if mul is not None:
        v, E = v * mul.double(), E * mul.double().abs()
    if residual is not None:
        v = v + residual.double()
    # one fp32 rounding of the sum, one of bf16
    tol = E + (v.abs() + E) * (BF16_HALF + 2.0 ** -22) + 2.0 ** -133
    err = (got.double() - v).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), got.double()[bad][0].item(),
                           v[bad][0].item(), tol[bad][0].item())
