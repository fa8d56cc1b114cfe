"""The int8 layer on every form of its kernels: split streaming, unsplit
streaming (straight stores and staged ones), CTA pairs in both orientations.
The cases name the form that they are meant for, and test_i8_forms_plan checks
that they are planned so."""
import math

import pytest
import torch

import i8ref
import rank_fp8_residual_b200 as ll
from test_gpu_i8 import _block, _check_product, _forward, _layer, _product_inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# (N, K) of a layer -> tokens per form
SPLIT, DIRECT, STAGED, PAIR, SWAP = "split", "direct", "staged", "pair", "swap"
NARROW = (2056, 2064)
WIDE = (16392, 4096)
FORMS = {NARROW: {SPLIT: 20, PAIR: 300}, WIDE: {DIRECT: 5, STAGED: 40, SWAP: 300, PAIR: 512}}
CASES = [(nk, form, M) for nk, forms in FORMS.items() for form, M in forms.items()]


# Shapes (M, K, N) with a part of a tile left over in every direction
REMAINDERS = {SPLIT: [(20, 2064, 2056), (100, 8208, 2056)], DIRECT: [(31, 1040, 18936), (5, 4112, 16392)],
              STAGED: [(40, 4112, 16392), (77, 1040, 18936), (130, 144, 18936)],
              PAIR: [(300, 2064, 2056), (513, 1040, 18936), (1025, 528, 3000)],
              SWAP: [(300, 4112, 16392), (80, 2064, 8200), (257, 1040, 18936)]}
# Feed-forwards (M, K, F) whose first product is of a form
STEPS = {SPLIT: (20, 512, 1536), DIRECT: (3, 512, 18944), STAGED: (40, 512, 18944), PAIR: (200, 512, 18944),
         SWAP: (257, 1040, 18944)}


def form_of(N, K, M, num_sms=148):
    kernel, _, tokens, splits = ll.ll_i8_plan(N, K, M, num_sms)
    if kernel == ll.LL_I8_STREAM:
        return SPLIT if splits > 1 else STAGED if tokens > 32 else DIRECT
    return SWAP if kernel == ll.LL_I8_PAIR_SWAP else PAIR


@pytest.mark.parametrize("nk", list(FORMS))
def test_a_row_does_not_depend_on_its_batch(nk):
    """The same tokens as the first and the last of batches of every form: the
    same bits."""
    N, K = nk
    xq, xs, wq, ws, b = _product_inputs(512, K, N, 7)
    layer = _layer(wq, ws, b)
    want = None
    for M in FORMS[nk].values():
        n = min(M, 16)
        got = _forward(layer, xq[:M], xs[:M])[:n]
        last = _forward(layer, xq[:M].flip(0), xs[:M].flip(0))[M - n:].flip(0)
        assert torch.equal(got, last)
        if want is None:
            want = got
        n = min(n, want.shape[0])
        assert torch.equal(got[:n], want[:n]), f"{M} tokens: {int((got[:n] != want[:n]).sum())} outputs differ"
        want = got if got.shape[0] > want.shape[0] else want


def _far_scales(M, N):
    """Token scales up to the 2^96 that the layer takes, feature scales anywhere
    in binary32."""
    xe = torch.tensor([7.9e28, 1.0, 2.0 ** -149, 1e-30, -1e28, 2.0 ** -120, 1e-10, 7e28])
    we = torch.tensor([1e33, 1e-30, 2.0 ** -140, 1e-38, 2.0 ** 120, -3.4e38, 1.0, 3e-45])
    return xe[torch.arange(M) % 8], we[torch.arange(N) % 8]


@pytest.mark.parametrize("nk,form,M", CASES)
def test_scales_far_from_one_on_every_form(nk, form, M):
    """Scales of features far from 1 meet sums that their tokens' scales have
    brought back, or not: (sum, scale of the token, of the feature) = (1e6, 1e-30,
    1e33) is 1e9 although the sum times 1e33 is beyond binary32.  Infinite where
    the output is beyond bf16, the bias where the sum is zero."""
    N, K = nk
    g = torch.Generator().manual_seed(M)
    xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    xq[0] = 0
    n = 64  # features, repeated: the reference needs no more
    wq = torch.randint(-128, 128, (n, K), generator=g, dtype=torch.int8)
    xs, ws = _far_scales(M, n)
    assert xs.abs().max() < 2.0 ** 96 < 1.01 * xs.abs().max()
    b = torch.randn(n, generator=g).to(BF16)
    reps = (N + n - 1) // n
    layer = _layer(wq.repeat(reps, 1)[:N].contiguous(), ws.repeat(reps)[:N].contiguous(), b.repeat(reps)[:N].contiguous())
    y = _forward(layer, xq, xs).cpu()
    for first in (0, (N // n - 1) * n):
        part = y[:, first:first + n].double()
        ref, size = i8ref.product(xq, xs, wq, ws, b, False)
        far = ref.abs() > 3.4e38
        assert far.any() and (~far).any()
        assert torch.isinf(part[far]).all() and torch.equal(part[far] > 0, ref[far] > 0)
        near = ref.abs() < 3.3e38  # between the two, rounding decides
        i8ref.check_y(part[near], ref[near], i8ref.PRODUCT_TOL * size[near], form)
        assert torch.equal(part[0], b.double())


@pytest.mark.parametrize("nk,form,M", CASES)
def test_waits_that_run_out_while_the_loads_arrive(nk, form, M):
    """With a limit of a nanosecond any wait may give up while the kernel's own
    loads and products are on their way: it lets them end, tells so, and the layer
    works on.  (What such a forward gives is not looked at.)"""
    N, K = nk
    xq, xs, wq, ws, b = _product_inputs(M, K, N, 9)
    layer = _layer(wq, ws, b)
    want = _forward(layer, xq, xs)
    x, s = xq.cuda(), xs.cuda()
    for _ in range(3):
        ll.ll_i8_set_debug(layer.handle, False, 1)
        for _ in range(4):
            layer.forward(x, s)
        torch.cuda.synchronize()
        assert ll.ll_i8_status(layer.handle) in (ll.LL_OK, ll.LL_ERR_DEVICE_TIMEOUT)
        ll.ll_i8_set_debug(layer.handle, False, 2_000_000_000)
        assert torch.equal(_forward(layer, xq, xs), want)


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("form,shape", [(f, s) for f, shapes in REMAINDERS.items() for s in shapes])
def test_product_with_remainders(form, shape, gelu):
    _check_product(*shape, bias=not gelu or form != PAIR, gelu=gelu, seed=sum(shape))


@pytest.mark.parametrize("nk,form,M", CASES)
def test_withheld_loads_time_out_on_every_form(nk, form, M):
    N, K = nk
    xq, xs, wq, ws, b = _product_inputs(M, K, N, 10)
    layer = _layer(wq, ws, b)
    want = _forward(layer, xq, xs)
    x, s = xq.cuda(), xs.cuda()
    ll.ll_i8_set_debug(layer.handle, True, 1_000_000)
    layer.forward(x, s)
    torch.cuda.synchronize()
    assert ll.ll_i8_status(layer.handle) == ll.LL_ERR_DEVICE_TIMEOUT
    ll.ll_i8_set_debug(layer.handle, False, 2_000_000_000)
    assert torch.equal(_forward(layer, xq, xs), want)


@pytest.mark.parametrize("nk,form,M", CASES)
def test_nan_scales_on_every_form(nk, form, M):
    N, K = nk
    xq, xs, wq, ws, b = _product_inputs(M, K, N, 11)
    layer = _layer(wq, ws, b, gelu=True)
    want = _forward(layer, xq, xs).cpu()
    for m in (0, M // 2, M - 1):
        bad = xs.clone()
        bad[m] = math.nan
        y = _forward(layer, xq, bad).cpu()
        assert torch.isnan(y[m]).all()
        keep = torch.arange(M) != m
        assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("form", list(STEPS))
def test_steps_one_by_one_back_to_back_and_replayed(form):
    """Steps of a feed-forward whose first product is of the form, each kernel
    allowed to start under the end of the one before: the same bits as with a
    wait after every call."""
    M, K, F = STEPS[form]
    results = []
    for mode in range(3):
        t, step = _block(M, K, F, 81)
        torch.cuda.synchronize()
        if mode == 0:
            for _ in range(12):
                step(torch.cuda.synchronize)
        elif mode == 1:
            for _ in range(12):
                step()
        else:
            h0, d0 = t["h"].clone(), t["d"].clone()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for _ in range(6):
                    step()
            t["h"].copy_(h0)
            t["d"].copy_(d0)
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        results.append((t["h"].cpu(), t["d"].cpu()))
    for r in results[1:]:
        assert torch.equal(r[0], results[0][0]) and torch.equal(r[1], results[0][1])
    assert torch.isfinite(results[0][0].float()).all()


@pytest.mark.parametrize("nk,form,M", CASES)
def test_one_layer_on_two_streams_and_in_two_graphs(nk, form, M):
    """Forwards of a layer on two streams at once, each with its own tokens."""
    N, K = nk
    xq, xs, wq, ws, b = _product_inputs(2 * M, K, N, 12)
    layer = _layer(wq, ws, b)
    want = [_forward(layer, xq[k * M:(k + 1) * M], xs[k * M:(k + 1) * M]) for k in range(2)]
    dev = [(xq[k * M:(k + 1) * M].cuda(), xs[k * M:(k + 1) * M].cuda()) for k in range(2)]
    outs = [torch.zeros(M, N, dtype=BF16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(15):
        for k in range(2):
            layer.forward(*dev[k], out=outs[k], stream=streams[k])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[k]):
            for _ in range(3):
                layer.forward(*dev[k], out=outs[k])
        graphs.append(g)
        outs[k].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for k, g in enumerate(graphs):
            with torch.cuda.stream(streams[k]):
                g.replay()
    torch.cuda.synchronize()
    assert ll.ll_i8_status(layer.handle) == ll.LL_OK
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
