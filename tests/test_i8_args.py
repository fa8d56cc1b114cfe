"""Refusals of the int8 operators before any device work: they are decided on
the host from sizes, alignment and address ranges, so no GPU is needed (the
addresses below are never read)."""
import math

import pytest
import torch

import i8ref
import rank_fp8_residual_b200 as ll

A, B, C, D, E = (0x10_0000_0000 + i * 0x1_0000_0000 for i in range(5))


def _code(fn, *args):
    with pytest.raises(ll.LLError) as e:
        fn(*args)
    return e.value.code


def _norm(x=A, residual=None, weight=None, eps=1e-6, M=4, K=64, h=None, y=None, codes=C, scale=D):
    return ll.ll_rmsnorm_i8(x, residual, weight, eps, M, K, h, y, codes, scale, 0)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(K=0), dict(K=8), dict(K=72), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan),
    dict(eps=math.inf), dict(x=None), dict(scale=None), dict(codes=None), dict(codes=None, scale=None),
    dict(h=B), dict(x=A + 2), dict(residual=B + 8), dict(weight=B + 8), dict(residual=B, h=E + 8), dict(y=E + 8),
    dict(codes=C + 8), dict(scale=D + 2),
    dict(codes=A), dict(y=A), dict(residual=B, y=B), dict(scale=A + 64), dict(weight=C), dict(y=C),
    dict(residual=B, h=A + 16), dict(residual=B, h=C), dict(scale=C + 64), dict(residual=B, h=E, y=E + 128)])
def test_norm_refuses(change):
    assert _code(lambda: _norm(**change)) == ll.LL_ERR_INVALID_ARG


def test_norm_row_limit_and_empty_batch():
    assert _code(lambda: _norm(K=65552)) == ll.LL_ERR_UNSUPPORTED
    _norm(M=0)
    _norm(M=0, x=None, codes=None, scale=None)  # an empty tensor's address is null
    ll.ll_quantize_i8(A, 0, 64, C, D, 0)
    assert _code(ll.ll_quantize_i8, A, 4, 65552, C, D, 0) == ll.LL_ERR_UNSUPPORTED


@pytest.mark.parametrize("args", [(A, -1, 64, C, D), (A, 4, 8, C, D), (A, 4, 40, C, D), (None, 4, 64, C, D),
                                  (A, 4, 64, None, D), (A, 4, 64, C, None), (A + 2, 4, 64, C, D), (A, 4, 64, C + 8, D),
                                  (A, 4, 64, C, D + 1), (A, 4, 64, A, D), (A, 4, 64, C, A + 16), (A, 4, 64, C, C + 16)])
def test_quantize_refuses(args):
    assert _code(ll.ll_quantize_i8, *args, 0) == ll.LL_ERR_INVALID_ARG


@pytest.mark.parametrize("N,K", [(0, 64), (7, 64), (-8, 64), (8, 0), (8, 8), (8, 24)])
def test_layer_create_refuses(N, K):
    assert _code(ll.ll_i8_create, N, K) == ll.LL_ERR_INVALID_ARG


def test_layer_reduction_limit():
    assert _code(ll.ll_i8_create, 8, 131072) == ll.LL_ERR_UNSUPPORTED
    # the largest sum of products of codes, -128 * -128 each, fits int32
    assert 131056 * 128 * 128 < 2 ** 31 <= 131072 * 128 * 128


def test_limit_of_the_rows():
    """A tile that starts at the last row still counts its rows in an int."""
    assert _code(ll.ll_i8_create, 2 ** 31 - 504, 16) == ll.LL_ERR_UNSUPPORTED
    assert _code(ll.ll_i8_plan, 2 ** 31 - 504, 16, 1, 148) == ll.LL_ERR_UNSUPPORTED
    assert _code(ll.ll_i8_plan, 8, 16, 2 ** 31 - 511, 148) == ll.LL_ERR_UNSUPPORTED
    assert ll.ll_i8_plan(8, 16, 2 ** 31 - 512, 148)[0] != ll.LL_I8_STREAM
    assert ll.ll_i8_plan(2 ** 31 - 512, 16, 1, 148)[0] == ll.LL_I8_STREAM


def test_null_layer_is_refused():
    for fn in (lambda: ll.ll_i8_forward(None, A, B, C, 4, 0), lambda: ll.ll_i8_set_weights(None, A, B),
               lambda: ll.ll_i8_set_epilogue(None, 0), lambda: ll.ll_i8_set_debug(None, False, 1)):
        assert _code(fn) == ll.LL_ERR_INVALID_ARG
    assert ll.ll_i8_status(None) == ll.LL_ERR_INVALID_ARG
    ll.ll_i8_destroy(None)


def test_tensors_are_checked_before_their_addresses_are_taken():
    """Host tensors, other types, shapes and strides never reach the library."""
    x, codes, scale = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    assert _code(ll.ll_quantize_i8, x, 4, 64, codes, scale, 0) == ll.LL_ERR_INVALID_ARG
    assert _code(ll.ll_rmsnorm_i8, x, None, None, 1e-6, 4, 64, None, None, codes, scale, 0) == ll.LL_ERR_INVALID_ARG


def test_reference_codes_round_ties_to_even_and_mark_bad_rows():
    u = torch.tensor([[254.0, 1.0, 3.0, 5.0, -1.0, -3.0], [0.0] * 6, [1.0, math.inf, 0, 0, 0, 0],
                      [1.0, math.nan, 0, 0, 0, 0]])
    codes, a = i8ref.codes_of(u)
    assert codes[0].tolist() == [127, 0, 2, 2, 0, -2]
    assert codes[1:].abs().sum() == 0
    assert a[0] == 254.0 and a[1] == 0.0 and math.isnan(a[2]) and math.isnan(a[3])
