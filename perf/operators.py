"""Cases of the int8 operators: the RMS norm with the residual's addition and an int8 output
(``ll_rmsnorm_i8``), the per-row int8 quantisation (``ll_quantize_i8``) and the int8 matrix product
with scales for each token and output feature (``Int8LinearLayer``).

With ``own`` false ``run`` computes the operators in plain torch operations; with ``own`` true it
calls this repository's kernels.  The int8 codes are whole numbers with one right value each (the
nearest integer of 127 u / max |u|, ties to the even one, where every u is exact in binary32), so
they are returned as they are, beside the scale that they are to be multiplied with.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
MAX_MK = 16384 * 4096          # values of the largest norm and quantisation
MAX_MNK = 16384 * 4096 * 16384  # multiply-adds of the largest product


def listed():
    return [
        # One token of a decoding step through the norm before a layer: latency.
        dict(name="norm_decode_m1_k4096", op="norm", M=1, K=4096, residual=True, weight=True, y=False),
        # The tokens of one 480x704x81 video latent before the attention projection.
        dict(name="norm_attn_m3630_k2048", op="norm", M=3630, K=2048, residual=True, weight=True, y=False),
        # A long prompt before a wide layer; the bf16 output feeds a bf16 layer beside the int8 one.
        dict(name="norm_long_m16384_k4096", op="norm", M=16384, K=4096, residual=True, weight=True, y=True),
        # A ragged batch through a norm without gain or residual (an adaptive norm's inner part).
        dict(name="norm_odd_m777_k5008", op="norm", M=777, K=5008, residual=False, weight=False, y=True),
        # The activations of a decoding batch before the second linear of a feed-forward.
        dict(name="quant_decode_m16_k8192", op="quant", M=16, K=8192),
        # A weight of the small-batch layer, quantised per output feature.
        dict(name="quant_weight_n16384_k4096", op="quant", M=16384, K=4096),
        # One token through the small-batch layer: the weight is read once.
        dict(name="product_m1_k4096_n16384", op="product", M=1, K=4096, N=16384, bias=True, gelu=False),
        # A decoding batch through the same layer.
        dict(name="product_m64_k4096_n16384", op="product", M=64, K=4096, N=16384, bias=True, gelu=False),
        # Odd sizes in every direction: partial tiles of tokens, features and the reduction.
        dict(name="product_odd_m333_k1040_n1000", op="product", M=333, K=1040, N=1000, bias=False, gelu=False),
        # The feed-forward pair of the video transformer.
        dict(name="product_up_m3630_k2048_n8192", op="product", M=3630, K=2048, N=8192, bias=True, gelu=True),
        dict(name="product_down_m3630_k8192_n2048", op="product", M=3630, K=8192, N=2048, bias=True, gelu=False),
        # The largest sweep point.
        dict(name="product_m16384_k4096_n16384", op="product", M=16384, K=4096, N=16384, bias=True, gelu=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "product", "product", "product"])
    if op == "product":
        while True:
            c = dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 64, 8192, 16), N=_log(rng, 64, 16384, 8),
                     bias=rng.random() < 0.5, gelu=rng.random() < 0.3)
            if c["M"] * c["N"] * c["K"] <= MAX_MNK:
                return c
    while True:
        c = dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 64, 16384, 16))
        if op == "norm":
            c.update(residual=rng.random() < 0.7, weight=rng.random() < 0.8, y=rng.random() < 0.5)
        if c["M"] * c["K"] <= MAX_MK:
            return c


def _activations(g, M, K):
    """A residual stream: unit variance, tokens of different loudness, a few loud channels."""
    dev = "cuda"
    x = torch.randn(M, K, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(M, 1, generator=g, device=dev))
    x *= torch.where(torch.rand(1, K, generator=g, device=dev) < 0.005, 12.0, 1.0)
    return x.to(torch.bfloat16)


def _codes(g, M, K):
    """int8 codes as a quantised normal row has them: standard deviation about 127 / 4."""
    return (torch.randn(M, K, generator=g, device="cuda") * 31.0).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev = "cuda"
    M, K = case["M"], case["K"]
    s = dict(case)
    if case["op"] == "product":
        N = case["N"]
        s["codes"] = _codes(g, M, K)
        s["scale"] = torch.rand(M, generator=g, device=dev) * 0.03 + 0.01
        s["w_codes"] = _codes(g, N, K)
        s["w_scale"] = (torch.rand(N, generator=g, device=dev) + 0.5) / (31.0 * math.sqrt(K))
        s["b"] = (torch.randn(N, generator=g, device=dev) * 0.1).to(torch.bfloat16) if case["bias"] else None
        s["out"] = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        if own:
            import rank_fp8_residual_b200 as ll
            layer = ll.Int8LinearLayer(N, K, ll.LL_EPILOGUE_GELU_TANH if case["gelu"] else ll.LL_EPILOGUE_NONE)
            layer.set_weights(s["w_codes"], s["w_scale"], s["b"])
            s["layer"] = layer
        return s
    s["x"] = _activations(g, M, K)
    s["codes"] = torch.empty(M, K, dtype=torch.int8, device=dev)
    s["scale"] = torch.empty(M, dtype=torch.float32, device=dev)
    if case["op"] == "norm":
        s["r"] = _activations(g, M, K) if case["residual"] else None
        s["w"] = (1.0 + 0.1 * torch.randn(K, generator=g, device=dev)).to(torch.bfloat16) if case["weight"] else None
        s["h_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y_out"] = torch.empty_like(s["x"]) if case["y"] else None
    return s


def _plain_codes(u):
    """Codes and max |u| of each row.  The quotients are taken in 64 bits: in 32 a value next to the
    border between two codes could fall on the wrong side."""
    a = u.abs().amax(dim=1, keepdim=True)
    t = (127.0 * u.double()) / torch.where(a > 0, a, torch.ones_like(a)).double()
    return torch.round(t).to(torch.int8), a[:, 0]


def _plain_norm(s):
    out = {}
    h = s["x"].float()
    if s["residual"]:
        # The residual stream is kept in bf16, and the norm is of the values kept.
        h16 = (h + s["r"].float()).to(torch.bfloat16)
        out["h"] = h16
        h = h16.float()
    rstd = torch.rsqrt((h * h).mean(dim=1) + EPS)
    u = h * s["w"].float() if s["weight"] else h
    if s["y"]:
        out["y"] = (u * rstd[:, None]).to(torch.bfloat16)
    out["codes"], a = _plain_codes(u)
    out["scale"] = a * rstd / 127.0
    return out


def _plain_product(s):
    acc = s["codes"].float() @ s["w_codes"].float().t()
    acc *= s["scale"][:, None]
    acc *= s["w_scale"]
    if s["bias"]:
        acc += s["b"].float()
    if s["gelu"]:
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (acc + 0.044715 * acc * acc * acc))
        acc = 0.5 * acc * (1.0 + t)
    return {"y": acc.to(torch.bfloat16)}


def run(state):
    s = state
    if own:
        import rank_fp8_residual_b200 as ll
        if s["op"] == "product":
            return {"y": s["layer"].forward(s["codes"], s["scale"], out=s["out"])}
        if s["op"] == "quant":
            ll.ll_quantize_i8(s["x"], s["M"], s["K"], s["codes"], s["scale"])
            return {"codes": s["codes"], "scale": s["scale"]}
        ll.ll_rmsnorm_i8(s["x"], s["r"], s["w"], EPS, s["M"], s["K"], s["h_out"], s["y_out"], s["codes"], s["scale"])
        out = {"codes": s["codes"], "scale": s["scale"]}
        if s["residual"]:
            out["h"] = s["h_out"]
        if s["y"]:
            out["y"] = s["y_out"]
        return out
    if s["op"] == "product":
        return _plain_product(s)
    if s["op"] == "quant":
        codes, a = _plain_codes(s["x"].float())
        return {"codes": codes, "scale": a / 127.0}
    return _plain_norm(s)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "product":
        N = case["N"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * M + 4 * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if case["op"] == "quant":
        return {"bytes": 3 * M * K + 4 * M, "flops": 3 * M * K}
    per = 2 + 1 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
    return {"bytes": per * M * K + 4 * M + (2 * K if case["weight"] else 0), "flops": 6 * M * K}


def _exact_rows(u):
    """Codes by counting: the nearest integer of 127 |u| / a is the number of borders below it, found
    from the exact integers' comparison 254 |u| against (2 n + 1) a in 64 bits."""
    m, a = u.abs(), u.abs().max(dim=1, keepdim=True).values
    safe = torch.where(a > 0, a, torch.ones_like(a))
    n = torch.floor(127.0 * m / safe)
    rest = 254.0 * m - (2.0 * n + 1.0) * safe   # above the border when positive, on it when zero
    n = n + ((rest > 0) | ((rest == 0) & (n % 2 == 1))).double()
    return (torch.sign(u) * n).to(torch.int8), a[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        v = torch.matmul(s["codes"].double(), s["w_codes"].double().transpose(0, 1))
        v = v * (s["scale"].double()[:, None] * s["w_scale"].double()[None, :])
        if case["bias"]:
            v = v + s["b"].double()[None, :]
        if case["gelu"]:
            # 1 + tanh(z) = 2 / (1 + exp(-2 z))
            v = v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v.pow(3))))
        return {"y": v}
    if case["op"] == "quant":
        codes, a = _exact_rows(s["x"].double())
        return {"codes": codes, "scale": a / 127.0}
    out = {}
    h = s["x"].double()
    if case["residual"]:
        h = (h + s["r"].double()).to(torch.bfloat16)
        out["h"] = None  # rounded to bf16 as the sum is kept: the plain form's value is the exact one
        h = h.double()
    rms = torch.sqrt(h.pow(2).sum(dim=1) / case["K"] + EPS)
    u = h * s["w"].double()[None, :] if case["weight"] else h
    if case["y"]:
        out["y"] = u / rms[:, None]
    out["codes"], a = _exact_rows(u)
    out["scale"] = a / (rms * 127.0)
    return out
