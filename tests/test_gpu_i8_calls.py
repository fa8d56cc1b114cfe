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


def _layers():
    from synth_inputs import make_inputs
    ins = _product_inputs(40, 512, 264, 5)
    inp = make_inputs(40, 512, 264, 16, seed=6)
    lite = ll.LiteLinearLayer(264, 512, 16, inp.scale_mode)
    lite.set_weights(inp.A.cuda(), inp.B.cuda(), inp.Q.cuda(), inp.scale.cuda(), inp.bias.cuda())
    return [(_layer(*ins[2:]), (ins[0].cuda(), ins[1].cuda())), (lite, (inp.x.cuda(),))]


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("as_handle", [False, True])
def test_a_new_output_of_another_stream(which, as_handle):
    """An output made for a forward on another stream is not memory that the
    current stream still writes, nor does a later one take it over while the
    current stream still reads it."""
    layer, args = _layers()[which]
    want = layer.forward(*args)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_handle else side
    torch.cuda.synchronize()
    before = torch.empty_like(want)
    torch.cuda._sleep(100_000_000)  # keeps the current stream busy for some 50 ms
    before.fill_(7.0)
    taken = before.data_ptr()
    del before
    out = layer.forward(*args, stream=stream)
    assert out.data_ptr() != taken
    side.synchronize()
    assert torch.equal(out.cpu(), want.cpu())
    torch.cuda._sleep(100_000_000)
    copy, taken = out.clone(), out.data_ptr()
    del out
    again = layer.forward(*args, stream=stream)
    assert again.data_ptr() != taken
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and torch.equal(again, want)


@pytest.mark.parametrize("which", [0, 1])
def test_a_new_output_of_a_captured_forward(which):
    layer, args = _layers()[which]
    want = layer.forward(*args)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out = layer.forward(*args, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        copy = out.clone()
    for _ in range(2):
        out.zero_()
        copy.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(copy, want)


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_new_outputs_of_the_streams_that_have_a_number(handle):
    """The default stream, as 0 and as cudaStreamLegacy, and cudaStreamPerThread."""
    layer, args = _layers()[0]
    want = layer.forward(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = layer.forward(*args, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_streams_given_as_zero_and_as_the_current_one():
    layer, args = _layers()[0]
    want = layer.forward(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [layer.forward(*args, stream=side), layer.forward(*args)]
        torch.cuda.synchronize()
        got.append(layer.forward(*args, stream=0))
        torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)


def test_a_low_rank_layer_takes_no_limit_below_that_of_copies_in_flight():
    layer, args = _layers()[1]
    want = layer.forward(*args)
    ll.ll_set_debug(layer.handle, False, 1)
    got = [layer.forward(*args) for _ in range(3)]
    torch.cuda.synchronize()
    assert ll.ll_status(layer.handle) == ll.LL_OK
    assert all(torch.equal(t, want) for t in got)


def test_dense_weights_beyond_the_quantisations_rows_are_refused():
    W = torch.zeros(8, 65552, dtype=BF16, device="cuda")
    assert _code(lambda: ll.Int8LinearLayer.from_dense(W)) == ll.LL_ERR_UNSUPPORTED
    W = W[:, :65536].contiguous()
    W[:, 0] = 1.0
    c, s = torch.ones(1, 65536, dtype=torch.int8, device="cuda"), torch.ones(1, device="cuda")
    assert torch.equal(ll.Int8LinearLayer.from_dense(W).forward(c, s).cpu(), torch.ones(1, 8, dtype=BF16))
