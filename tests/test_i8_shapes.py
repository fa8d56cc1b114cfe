"""Shapes that the int8 operators' arguments may have.  The library sees
addresses only, so the binding tells a matrix from its transpose; stand-ins
replace the tensors, as the check comes before any address is used."""
import pytest
import torch

import rank_fp8_residual_b200 as ll


class _Tensor:
    """What the binding asks of a CUDA tensor."""
    dtype, is_cuda, device = torch.bfloat16, True, "cuda:0"

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def _taken(shape, M, K):
    try:
        return ll._buffer(_Tensor(*shape), "x", torch.bfloat16, M * K, None if M == 1 else (M, K)) == 4096
    except ll.LLError as e:
        assert e.code == ll.LL_ERR_INVALID_ARG
        return False


@pytest.mark.parametrize("shape,M,K", [
    ((8, 64), 8, 64), ((2, 4, 64), 8, 64), ((8, 4, 16), 8, 64), ((2, 4, 4, 16), 8, 64),  # split dimensions
    ((512,), 8, 64), ((64,), 1, 64), ((1, 64), 1, 64), ((64, 1), 1, 64),                 # flat, one row
    ((2, 256), 8, 64), ((16, 32), 8, 64),                                                # groups of a row, rows joined
    ((64, 64), 64, 64), ((0, 64), 0, 64), ((64, 0), 0, 64), ((0,), 0, 64), ((1, 1, 8, 64), 8, 64)])
def test_shapes_that_stand_for_the_rows(shape, M, K):
    ll._load_dtypes()
    assert _taken(shape, M, K)


@pytest.mark.parametrize("shape,M,K", [((64, 8), 8, 64), ((64, 2, 4), 8, 64), ((4, 16, 8), 8, 64), ((1, 64, 8), 8, 64),
                                       ((64, 8, 1), 8, 64), ((8, 32), 8, 64), ((9, 64), 8, 64), ((64,), 8, 64)])
def test_transposed_and_wrong_shapes_are_refused(shape, M, K):
    ll._load_dtypes()
    assert not _taken(shape, M, K)


def test_vectors_are_counted():
    ll._load_dtypes()
    for shape in ((8,), (8, 1), (2, 4)):
        assert ll._buffer(_Tensor(*shape), "scale", torch.bfloat16, 8) == 4096
    with pytest.raises(ll.LLError):
        ll._buffer(_Tensor(9), "scale", torch.bfloat16, 8)


@pytest.mark.parametrize("codes,scale,out", [
    ((8, 64), (8,), (8, 24)), ((8, 64), (8, 1), (8, 24)), ((2, 4, 64), (2, 4), (2, 4, 24)),
    ((2, 4, 64), (2, 4, 1), (2, 4, 24)), ((8, 1, 64), (8, 1), (8, 1, 24)), ((64,), (), (24,)), ((64,), (1,), (1, 24)),
    ((512,), (2, 4), (2, 4, 24)), ((8, 4, 16), (8,), (8, 24)), ((1, 64), (1, 1), (1, 24)), ((0, 64), (0, 1), (0, 24))])
def test_shape_of_a_forward(monkeypatch, codes, scale, out):
    """The leading dimensions of the scales, without one that a maximum kept."""
    calls = []

    class Lib:
        ll_i8_forward = staticmethod(lambda *a: calls.append(a) or 0)
        ll_i8_destroy = staticmethod(lambda h: None)

    monkeypatch.setattr(ll, "_lib", Lib)
    monkeypatch.setattr(ll, "_buffer", lambda t, *a: t)
    monkeypatch.setattr(ll, "_stream", lambda s: 0)
    layer = object.__new__(ll.Int8LinearLayer)
    layer.handle, layer.N, layer.K = 1, 24, 64
    try:
        y = layer.forward(torch.empty(codes, dtype=torch.int8), torch.empty(scale))
    finally:
        layer.handle = None  # never the library's
    assert y.shape == torch.Size(out) and y.dtype == torch.bfloat16
    assert calls[0][3] is y and calls[0][4] == y.numel() // 24
