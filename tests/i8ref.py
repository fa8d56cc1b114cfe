"""The int8 operators in 64 bits on the CPU, from their definitions, and the
tolerances of the GPU results.

Tolerances.  Codes have one right value: no tolerance.  h is one correctly
rounded sum: no tolerance.  scale and y go through rstd: the sum of squares
has positive terms (each exact in binary32), so with at most 64 added per
thread and 10 more levels across the block it is within 74 * 2^-24 of its
value, rstd within half of that; the division by K, the addition of eps, the
square root, the reciprocal, the product with a and the division by 127 add
at most 2^-24 each: 37 + 6 = 43, taken as 48 * 2^-24.  y is then rounded to
bf16, half a step or 2^-8 of its value.  The product's sum is exact; its
conversion, the product of the scales, their multiplication and the bias add
at most 4 * 2^-24 of |product| + |bias|; GELU has a slope of at most 1.13 and
its evaluation (a cubic, tanh or exp, two products) stays within 10 * 2^-24
of |v|: together under 16 * 2^-24 = 2^-20 of |product| + |bias|."""
import math

import torch

RSTD_TOL = 48 * 2.0 ** -24
BF16_HALF_STEP = 2.0 ** -8
PRODUCT_TOL = 2.0 ** -20
TINY = 2.0 ** -134  # half a step of the smallest bf16 subnormals


def codes_of(u):
    """Codes and a of rows u (float64, CPU)."""
    u = u.to(torch.float64)
    a = u.abs().amax(dim=1, keepdim=True)
    bad = ~torch.isfinite(u).all(dim=1, keepdim=True)
    q = 127.0 * u / torch.where((a > 0) & ~bad, a, torch.ones_like(a))
    codes = torch.where(bad, torch.zeros_like(q), torch.round(q)).to(torch.int8)
    return codes, torch.where(bad, torch.full_like(a, math.nan), a)[:, 0]


def rmsnorm(x, residual, weight, eps):
    """(h bf16, y float64, codes int8, scale float64)."""
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    hd = h.to(torch.float64)
    rstd = 1.0 / torch.sqrt(hd.pow(2).mean(dim=1) + eps)
    u = hd if weight is None else hd * weight.to(torch.float64)
    codes, a = codes_of(u)
    return h, u * rstd[:, None], codes, a * rstd / 127.0


def gelu_tanh(v):
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))


def product(codes, scale, w_codes, w_scale, bias, gelu):
    """(y float64, |product| + |bias| float64)."""
    p = (codes.to(torch.float64) @ w_codes.to(torch.float64).t()) * scale.to(torch.float64)[:, None]
    p = p * w_scale.to(torch.float64)[None, :]
    b = torch.zeros(w_codes.shape[0], dtype=torch.float64) if bias is None else bias.to(torch.float64)
    v = p + b
    return (gelu_tanh(v) if gelu else v), p.abs() + b.abs()


def check_scale(got, ref, what=""):
    got, nan = got.cpu().to(torch.float64), torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), what
    err = (got - ref)[~nan].abs()
    assert torch.all(err <= RSTD_TOL * ref[~nan].abs() + 2.0 ** -149), (what, float(err.max()))


def check_y(got, ref, extra, what=""):
    """|got - ref| <= half a bf16 step of ref and `extra` (before the
    rounding, so the half step is of a value that much larger)."""
    got = got.cpu().to(torch.float64)
    bound = BF16_HALF_STEP * (ref.abs() + extra) + extra + TINY
    bad = (got - ref).abs() > bound
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {ref[bad][0]}")
