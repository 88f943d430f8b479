"""Timed cases of the operators that stand around a W4 + Error Compensator layer in a serving step.

Four operators: the root-mean-square norm with the residual's addition (bf16 and / or 8-bit
output), the 8-bit quantisation of activations, the layer with bias, activation, multiplier and
residual in its epilogue on bf16 activations, and the same on 8-bit activations.

Formulas (t: token, n: output feature, k: input feature, j: rank):

  norm      h = bf16(x + residual),  v[t,k] = h[t,k] w[k] / sqrt(mean_k h[t,k]^2 + eps)
  quantise  a = max(max_k |v[t,k]|, 2^-100),  s[t] = a / 448,  q[t,k] = e4m3(v[t,k] * (448 / a))
  layer     Y[t,n] = sum_k x[t,k] s[n] (q[n,k] - z[n]) + g_t sum_j (sum_k x[t,k] A[k,j]) B[j,n],
            g_t = 1 / (1 + exp(-(x[t,:] . w_g + b_g)))
  epilogue  y = act(Y + bias) * mul + residual

`own` False computes them from elementary torch operations, `own` True through the package.
"""
import math

import torch

own = False

EPS = 1e-6
FLOOR = 2.0 ** -100
# the most multiply-adds of a drawn layer case: those of the largest listed one
MOST_MACS = 4096 * 4096 * 14336
MOST_ELEMENTS = 8192 * 4096


def listed():
    return [
        # one sequence being decoded, hidden size 4096: the norm in front of the q/k/v projections
        {"name": "norm 1x4096", "op": "norm", "M": 1, "K": 4096, "residual": True, "bf16": True, "q8": False},
        # a small ragged batch, row length no multiple of a vector load
        {"name": "norm q8 37x2050", "op": "norm", "M": 37, "K": 2050, "residual": True, "bf16": True, "q8": True},
        # a prefill batch whose next layer takes 8-bit activations
        {"name": "norm q8 8192x4096", "op": "norm", "M": 8192, "K": 4096, "residual": True, "bf16": False, "q8": True},
        # the MLP's inner activations in front of the down projection: a decode batch ...
        {"name": "quant 16x14336", "op": "quant", "M": 16, "K": 14336},
        # ... and a prefill batch with a ragged token count
        {"name": "quant 2047x14336", "op": "quant", "M": 2047, "K": 14336},
        # o projection of one decoded token, added to the residual stream
        {"name": "ep o 1x4096x4096", "op": "ep", "M": 1, "K": 4096, "N": 4096, "r": 32, "asym": False, "act": "none",
         "bias": False, "mul": False, "residual": True},
        # a small batch on a narrow layer with odd sizes, min-max quantised, biased
        {"name": "ep 19x1032x2744", "op": "ep", "M": 19, "K": 1032, "N": 2744, "r": 8, "asym": True, "act": "gelu",
         "bias": True, "mul": False, "residual": False},
        # MLP up projection of a prefill batch, times the activated gate projection
        {"name": "ep up 2048x4096x14336", "op": "ep", "M": 2048, "K": 4096, "N": 14336, "r": 64, "asym": False,
         "act": "none", "bias": False, "mul": True, "residual": False},
        # q projection of four decoded tokens on 8-bit activations
        {"name": "q8 q 4x4096x4096", "op": "q8", "M": 4, "K": 4096, "N": 4096, "r": 32, "asym": False, "act": "none",
         "bias": True, "mul": False, "residual": False},
        # MLP down projection of a decode batch, added to the residual stream
        {"name": "q8 down 64x14336x4096", "op": "q8", "M": 64, "K": 14336, "N": 4096, "r": 64, "asym": False,
         "act": "none", "bias": False, "mul": False, "residual": True},
        # a ragged chunk on a narrow layer of odd sizes, min-max quantised
        {"name": "q8 333x2064x1000", "op": "q8", "M": 333, "K": 2064, "N": 1000, "r": 24, "asym": True,
         "act": "gelu_tanh", "bias": True, "mul": False, "residual": True},
        # MLP gate projection of a prefill batch with its activation
        {"name": "q8 gate 4096x4096x14336", "op": "q8", "M": 4096, "K": 4096, "N": 14336, "r": 64, "asym": False,
         "act": "silu", "bias": False, "mul": False, "residual": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "ep", "ep", "q8", "q8"])
    if op in ("norm", "quant"):
        K = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            K = max(64, K // 8 * 8)
        M = _log(rng, 1, max(2, min(8192, MOST_ELEMENTS // K)))
        if op == "quant":
            return {"op": op, "M": M, "K": K}
        q8 = rng.random() < 0.6
        return {"op": op, "M": M, "K": K, "residual": rng.random() < 0.7, "bf16": not q8 or rng.random() < 0.4,
                "q8": q8}
    K = max(256, _log(rng, 256, 14336) // 8 * 8)
    N = max(256, _log(rng, 256, 14336) // 8 * 8)
    M = _log(rng, 1, min(4096, MOST_MACS // (K * N)))
    return {"op": op, "M": M, "K": K, "N": N, "r": rng.choice([0, 8, 16, 32, 64, 100, 128]),
            "asym": rng.random() < 0.5, "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
            "bias": rng.random() < 0.5, "mul": rng.random() < 0.3, "residual": rng.random() < 0.5}


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _activations(gen, M, K):
    """N(0, 1) with one input channel in a hundred twenty times larger."""
    x = _normal(gen, M, K)
    hot = torch.rand(K, generator=gen, device="cuda") < 0.01
    return torch.where(hot, x * 20, x)


def _quantised_layer(gen, case):
    """4-bit codes, eight a word, with a scale and zero point a channel, and the Error Compensator."""
    K, N, r = case["K"], case["N"], case["r"]
    W = _normal(gen, N, K, std=0.02)
    if case["asym"]:
        W = W + _normal(gen, N, 1, std=0.01)
        lo, hi = W.amin(1, keepdim=True).clamp(max=0), W.amax(1, keepdim=True).clamp(min=0)
        s = (hi - lo) / 15
        z = (-lo / s).round().clamp(0, 15)
        q = ((W / s).round() + z).clamp(0, 15)
    else:
        s = W.abs().amax(1, keepdim=True) / 7
        z = torch.full_like(s, 8)
        q = (W / s).round().clamp(-8, 7) + 8
    q = q.to(torch.int32).view(N, K // 8, 8)
    codes = torch.zeros(N, K // 8, dtype=torch.int32, device="cuda")
    for i in range(8):
        codes |= q[:, :, i] << (4 * i)
    layer = {"codes": codes, "s": s.flatten().contiguous(), "z": z.flatten().to(torch.uint8), "A": None, "B": None,
             "w_g": None, "b_g": 0.0}
    if r:
        layer |= {"A": _normal(gen, K, r, std=0.01).bfloat16(), "B": _normal(gen, r, N, std=0.01).bfloat16(),
                  "w_g": _normal(gen, K, std=1 / math.sqrt(K)).bfloat16(), "b_g": -0.25}
    return layer


def _to_8_bits(v):
    a = v.abs().amax(1, keepdim=True).clamp(min=FLOOR)
    return (v * (448 / a)).to(torch.float8_e4m3fn), (a / 448).flatten()


def _case(case, seed):
    """The tensors that a serving step holds in front of the call."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    M, K = case["M"], case["K"]
    st = {"case": case, "x": _activations(gen, M, K).bfloat16()}
    if case["op"] == "norm":
        st["w"] = (1 + _normal(gen, K, std=0.1)).bfloat16()
        st["residual"] = _normal(gen, M, K).bfloat16() if case["residual"] else None
    elif case["op"] in ("ep", "q8"):
        N = case["N"]
        st["layer"] = _quantised_layer(gen, case)
        st["bias"] = _normal(gen, N, std=0.5).bfloat16() if case["bias"] else None
        st["mul"] = _normal(gen, M, N).bfloat16() if case["mul"] else None
        st["residual"] = _normal(gen, M, N).bfloat16() if case["residual"] else None
        if case["op"] == "q8":
            st["xq"], st["xs"] = _to_8_bits(st.pop("x").float())
    return st


def prepare(case, seed):
    st = _case(case, seed)
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        st["out"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda") if case["bf16"] else None
        st["h"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda") if case["residual"] else None
    elif case["op"] in ("ep", "q8"):
        st["out"] = torch.empty(M, case["N"], dtype=torch.bfloat16, device="cuda")
    if case["op"] == "quant" or case.get("q8"):
        st["q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        st["qs"] = torch.empty(M, dtype=torch.float32, device="cuda")
    if own and "layer" in st:  # the handle that a program loads its weights into
        from w4_gemm_error_b200.spear import W4ECLinear

        lay = st["layer"]
        st["handle"] = W4ECLinear(None, lay["A"], lay["B"], lay["w_g"], lay["b_g"], max_M=M,
                                  packed=(lay["codes"], lay["s"], lay["z"]))
    return st


def _activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain(st):
    case = st["case"]
    if case["op"] == "quant":
        q, s = _to_8_bits(st["x"].float())
        return {"q": q, "s": s}
    if case["op"] == "norm":
        h, got = st["x"], {}
        if case["residual"]:
            got["h"] = h = (h.float() + st["residual"].float()).bfloat16()
        v = h.float()
        v = v * (1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)) * st["w"].float()
        if case["bf16"]:
            got["y"] = v.bfloat16()
        if case["q8"]:
            got["q"], got["s"] = _to_8_bits(v)
        return got
    lay = st["layer"]
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device="cuda")
    q = ((lay["codes"].unsqueeze(2) >> shifts) & 15).view(lay["codes"].shape[0], -1)
    W = (q.float() - lay["z"].float()[:, None]) * lay["s"][:, None]
    x = st["xq"].float() * st["xs"][:, None] if case["op"] == "q8" else st["x"].float()
    v = x @ W.t()
    if case["r"]:
        g = 1 / (1 + torch.exp(-(x @ lay["w_g"].float() + lay["b_g"])))
        v = v + g[:, None] * ((x @ lay["A"].float()) @ lay["B"].float())
    if st["bias"] is not None:
        v = v + st["bias"].float()
    v = _activate(v, case["act"])
    if st["mul"] is not None:
        v = v * st["mul"].float()
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return {"y": v.bfloat16()}


def _called(st):
    case = st["case"]
    if case["op"] == "quant":
        from w4_gemm_error_b200.spear import quantize_q8

        q, s = quantize_q8(st["x"], out_q=st["q"], out_s=st["qs"])
        return {"q": q, "s": s}
    if case["op"] == "norm":
        from w4_gemm_error_b200.spear import rmsnorm

        y, q, s, h = rmsnorm(st["x"], st["w"], EPS, st["residual"], bf16=case["bf16"], q8=case["q8"], out=st["out"],
                             out_q=st.get("q"), out_s=st.get("qs"), out_sum=st["h"])
        got = {"h": h, "y": y, "q": q, "s": s}
        return {k: v for k, v in got.items() if v is not None}
    more = {"act": case["act"], "bias": st["bias"], "mul": st["mul"], "residual": st["residual"], "out": st["out"]}
    if case["op"] == "q8":
        return {"y": st["handle"].forward_q8(st["xq"], st["xs"], **more)}
    return {"y": st["handle"].forward_ep(st["x"], **more)}


def run(state):
    return _called(state) if own else _plain(state)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quant":
        return {"bytes": 3 * M * K + 4 * M, "flops": 2 * M * K}
    if case["op"] == "norm":
        b = 2 * M * K + 2 * K
        b += 4 * M * K if case["residual"] else 0
        b += 2 * M * K if case["bf16"] else 0
        b += M * K + 4 * M if case["q8"] else 0
        return {"bytes": b, "flops": 6 * M * K}
    N, r = case["N"], case["r"]
    b = N * K / 2 + 5 * N + 2 * M * N * (1 + case["mul"] + case["residual"]) + 2 * N * case["bias"]
    b += M * K + 4 * M if case["op"] == "q8" else 2 * M * K
    f = 2 * M * N * K
    if r:
        b += 2 * r * (K + N) + 2 * K
        f += 2 * M * (K * (r + 1) + r * N)
    return {"bytes": b, "flops": f}


def exact(case, seed):
    """The definitions in 64 bits. An 8-bit output has the value that its code rounds, in units of the row's scale."""
    st = _case(case, seed)
    x = st["xq"].double() * st["xs"].double().unsqueeze(1) if case["op"] == "q8" else st["x"].double()

    def codes(v):
        top = torch.maximum(v.abs().max(dim=1).values, torch.tensor(FLOOR, dtype=torch.float64, device="cuda"))
        return v / top.unsqueeze(1) * 448, top / 448

    if case["op"] == "quant":
        q, s = codes(x)
        return {"q": q, "s": s}
    if case["op"] == "norm":
        got = {}
        if case["residual"]:
            x = x + st["residual"].double()
            got["h"] = x
            x = x.to(torch.bfloat16).double()  # the norm is that of the sum as it is stored
        v = x / (x.pow(2).sum(1) / case["K"] + EPS).sqrt().unsqueeze(1) * st["w"].double()
        if case["bf16"]:
            got["y"] = v
        if case["q8"]:
            got["q"], got["s"] = codes(v)
        return got
    lay, M, N = st["layer"], case["M"], case["N"]
    words = lay["codes"].to(torch.int64)
    total = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for i in range(8):  # the input features 8 j + i
        d = ((words >> (4 * i)) & 15).double() - lay["z"].double().unsqueeze(1)
        total += x[:, i::8] @ d.t()
    total *= lay["s"].double()
    if case["r"]:
        gate = torch.sigmoid(x @ lay["w_g"].double() + lay["b_g"])
        total += gate.unsqueeze(1) * (x @ lay["A"].double() @ lay["B"].double())
    if case["bias"]:
        total += st["bias"].double()
    act = case["act"]
    if act == "relu":
        total = torch.where(total > 0, total, torch.zeros_like(total))
    elif act == "silu":
        total = total * torch.sigmoid(total)
    elif act == "gelu":
        total = total * 0.5 * torch.special.erfc(-total / math.sqrt(2.0))
    elif act == "gelu_tanh":  # 0.5 (1 + tanh(a)) = 1 / (1 + exp(-2 a))
        total = total * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (total + 0.044715 * total.pow(3)))
    if case["mul"]:
        total = total * st["mul"].double()
    if case["residual"]:
        total = total + st["residual"].double()
    return {"y": total}
