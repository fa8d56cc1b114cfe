"""The norm's bf16 output where it is not finite: rows with NaN and infinities,
gains with them, values beyond bf16.

A y of the definition that is beyond binary32's rounding to bf16 is infinite:
from 2^127 (2 - 2^-8) on, half a step above the largest bf16; within 2^-17 of
that border (more than i8ref.RSTD_TOL) either is right."""
import math

import pytest
import torch

import i8ref
import rank_fp8_residual_b200 as ll
from test_gpu_i8 import _norm, _rows, _special_rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
BORDER = 2.0 ** 127 * (2 - 2.0 ** -8)


def _check(x, r, w, eps=1e-6, **kw):
    h, y, codes, scale = _norm(x, r, w, eps, **kw)
    rh, ry, rc, rs = i8ref.rmsnorm(x, r, w, eps)
    y = y.double()
    nan = torch.isnan(ry)
    assert torch.equal(torch.isnan(y), nan)
    over = ry.abs() > BORDER * (1 + 2.0 ** -17)
    assert torch.equal(y[over], torch.sign(ry[over]) * math.inf)
    fine = ry.abs() < BORDER * (1 - 2.0 ** -17)
    i8ref.check_y(y[fine], ry[fine], i8ref.RSTD_TOL * ry[fine].abs(), "y")
    if h is not None:
        assert torch.equal(h.nan_to_num(0.5, 9.0, -9.0), rh.nan_to_num(0.5, 9.0, -9.0))
        assert torch.equal(torch.isnan(h), torch.isnan(rh))
    if codes is not None:
        assert torch.equal(codes, rc)
        i8ref.check_scale(scale, rs)
    return nan, over


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("K", [16, 512, 4096, 16400])
def test_y_of_rows_with_nan_or_infinity(K, codes):
    x = _rows(7, K, 12)
    x[1, 3] = math.nan
    x[2, K - 1] = math.inf
    x[4, 0] = -math.inf
    x[5, 0], x[5, 9] = math.inf, -math.inf
    r, w = _rows(7, K, 13), _rows(1, K, 14, 0.0)[0]
    for args in ((x, None, None), (x, None, w), (x, r, None), (x, r, w), (r, x, w)):
        for h in (True, False):
            nan, _ = _check(*args, h=h, codes=codes)
            assert nan.any(1).tolist() == [False, True, True, False, True, True, False] and nan[1].all()
            assert nan[2].sum() == 1 and nan[5].sum() == 2
    r = x.clone()
    r[2, K - 1] = -math.inf  # the infinities cancel to NaN
    assert _check(x, r, w, codes=codes)[0][2].all()


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("K", [16, 512, 4096, 16400])
def test_y_under_gains_with_nan_or_infinity(K, codes):
    x = _rows(4, K, 15)
    x[1] = 0.0
    w = torch.ones(K, dtype=BF16)
    w[5], w[6], w[7] = math.inf, -math.inf, math.nan
    nan, over = _check(x, None, w, codes=codes)
    assert nan[0].sum() == 1 and nan[1].sum() == 3 and over[0].sum() == 2
    _check(x, _rows(4, K, 16), w, codes=codes)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("K", [16, 512, 4096, 16400])
def test_y_beyond_bf16(K, codes):
    x = _special_rows(K)
    one = 1 + 0.2 * _rows(1, K, 42, 0.0)[0].float()
    w = (one.clamp(-1.9, 1.9) * 2.0 ** 127).to(BF16)
    for r in (None, torch.zeros_like(x)):
        _, over = _check(x, r, w, codes=codes)
        assert over.any() and not over.all()
    _check(x, x, w, eps=1e-30, codes=codes)
    x = torch.full((3, K), 3e38).to(BF16)  # h beyond bf16 itself
    _check(x, x, None, codes=codes)
