"""Calls of the int8 operators through the binding: shapes, streams, buffers."""
import pytest
import torch

import i8ref
import rank_fp8_residual_b200 as ll
from test_gpu_i8 import _layer, _product_inputs, _rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _code(fn):
    with pytest.raises(ll.LLError) as e:
        fn()
    return e.value.code


def test_transposed_matrices_are_refused():
    M, K, N = 8, 64, 24
    xq, xs, wq, ws, b = (t.cuda() for t in _product_inputs(M, K, N, 3))
    layer = _layer(wq, ws, b)
    want = layer.forward(xq, xs)
    x = _rows(M, K, 4).cuda()
    c, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    turn = lambda t: t.t().contiguous()  # noqa: E731
    for fn in (lambda: layer.forward(turn(xq), xs), lambda: layer.forward(xq, xs, out=turn(want)),
               lambda: layer.set_weights(turn(wq), ws, b), lambda: ll.ll_quantize_i8(turn(x), M, K, c, s),
               lambda: ll.ll_quantize_i8(x, M, K, turn(c), s),
               lambda: ll.ll_rmsnorm_i8(x, turn(x), None, 1e-6, M, K, None, None, c, s),
               lambda: ll.ll_rmsnorm_i8(x, None, None, 1e-6, M, K, None, turn(x), c, s)):
        assert _code(fn) == ll.LL_ERR_INVALID_ARG
    assert torch.equal(layer.forward(xq, xs), want)
    # heads x width, and groups of a row as rows of their own
    assert torch.equal(layer.forward(xq.view(M, 4, 16), xs), want)
    ll.ll_quantize_i8(x, 4 * M, K // 4, c, torch.empty(4 * M, device="cuda"))
    assert torch.equal(c.cpu().view(4 * M, K // 4), i8ref.codes_of(x.cpu().view(4 * M, K // 4))[0])
