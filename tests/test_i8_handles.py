"""The int8 layer's calls by handle check what they are given before the
library sees an address.  The library is replaced: no GPU is needed."""
import pytest
import torch

import rank_fp8_residual_b200 as ll

N, K, M, H = 24, 64, 8, 4096


class _Cuda:
    """A CPU tensor that says it is a CUDA one."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return True if name == "is_cuda" else getattr(self.t, name)


def _t(dtype, *shape):
    return _Cuda(torch.empty(shape, dtype=dtype))


@pytest.fixture
def calls(monkeypatch):
    calls = []

    class Lib:
        ll_status_string = ll._lib.ll_status_string
        ll_i8_create = staticmethod(lambda n, k: H)
        ll_i8_set_weights = staticmethod(lambda *a: calls.append(a) or 0)
        ll_i8_forward = staticmethod(lambda *a: calls.append(a) or 0)
        ll_i8_destroy = staticmethod(lambda h: calls.append(h))

    monkeypatch.setattr(ll, "_lib", Lib)
    monkeypatch.setattr(ll, "_i8_sizes", {}, raising=False)
    assert ll.ll_i8_create(N, K) == H
    return calls


def _refused(fn):
    with pytest.raises(ll.LLError) as e:
        fn()
    return e.value.code == ll.LL_ERR_INVALID_ARG


I8, F32, BF16 = torch.int8, torch.float32, torch.bfloat16


def test_forward_takes_the_first_rows_of_what_it_is_given(calls):
    for rows in (M, M + 3):
        c, s, y = _t(I8, rows, K), _t(F32, rows), _t(BF16, rows, N)
        ll.ll_i8_forward(H, c, s, y, M, 0)
        assert calls.pop() == (H, c.data_ptr(), s.data_ptr(), y.data_ptr(), M, 0)
    ll.ll_i8_forward(H, 16, 32, 48, M, 0)  # addresses as they are
    assert calls.pop() == (H, 16, 32, 48, M, 0)


@pytest.mark.parametrize("bad", [
    dict(c=_t(I8, M - 1, K)), dict(c=_t(torch.uint8, M, K)), dict(c=_t(BF16, M, K)), dict(c=torch.empty(M, K, dtype=I8)),
    dict(c=_Cuda(torch.empty(M, 2 * K, dtype=I8)[:, :K])), dict(s=_t(F32, M - 1)), dict(s=_t(torch.float64, M)),
    dict(s=_Cuda(torch.empty(2 * M)[::2])), dict(y=_t(F32, M, N)), dict(y=_t(BF16, M, N - 8)), dict(y=_t(BF16, M - 1, N))])
def test_forward_refuses(calls, bad):
    a = dict(dict(c=_t(I8, M, K), s=_t(F32, M), y=_t(BF16, M, N)), **bad)
    assert _refused(lambda: ll.ll_i8_forward(H, a["c"], a["s"], a["y"], M, 0)) and not calls


@pytest.mark.parametrize("bad", [dict(c=_t(I8, N, K - 16)), dict(c=_t(BF16, N, K)), dict(s=_t(F32, N - 1)),
                                 dict(s=_t(BF16, N)), dict(b=_t(F32, N)), dict(b=_t(BF16, 1))])
def test_set_weights_refuses(calls, bad):
    a = dict(dict(c=_t(I8, N, K), s=_t(F32, N), b=_t(BF16, N)), **bad)
    assert _refused(lambda: ll.ll_i8_set_weights(H, a["c"], a["s"], a["b"])) and not calls


def test_a_destroyed_layer_is_no_layer(calls):
    ll.ll_i8_destroy(H)
    assert calls == [H]
    assert _refused(lambda: ll.ll_i8_forward(H, 16, 32, 48, M, 0)) and _refused(lambda: ll.ll_i8_set_weights(H, 16, 32))
    assert calls == [H]
