"""The int8 operators on the GPU against their definitions in 64 bits
(tolerances and their derivation in i8ref)."""
import math

import pytest
import torch

import i8ref
import rank_fp8_residual_b200 as ll

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _rows(M, K, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))
    x[:, ::37] *= 9.0
    return x.to(BF16)


def _norm(x, r, w, eps=1e-6, h=True, y=True, codes=True, in_place=None, stream=None):
    """Runs the norm with poisoned outputs one row longer than asked for."""
    M, K = x.shape
    dev = [None if t is None else t.cuda() for t in (x, r, w)]
    out_h = torch.full((M + 1, K), 7.0, dtype=BF16, device="cuda") if h and r is not None else None
    out_y = torch.full((M + 1, K), 7.0, dtype=BF16, device="cuda") if y else None
    out_c = torch.full((M + 1, K), 77, dtype=torch.int8, device="cuda") if codes else None
    out_s = torch.full((M + 1,), 7.0, device="cuda") if codes else None
    cut = lambda t: None if t is None else t[:M]  # noqa: E731
    ht = cut(out_h)
    if in_place is not None and ht is not None:
        ht = dev[in_place]
    ll.ll_rmsnorm_i8(*dev, eps, M, K, ht, cut(out_y), cut(out_c), cut(out_s), stream)
    torch.cuda.synchronize()
    for t, v in ((out_h, 7.0), (out_y, 7.0), (out_c, 77), (out_s, 7.0)):
        assert t is None or torch.all(t[M] == v), "a row behind the last was written"
    return tuple(None if t is None else t.cpu() for t in (ht, cut(out_y), cut(out_c), cut(out_s)))


def _check_norm(x, r, w, eps=1e-6, **kw):
    h, y, codes, scale = _norm(x, r, w, eps, **kw)
    rh, ry, rc, rs = i8ref.rmsnorm(x, r, w, eps)
    if h is not None:
        assert torch.equal(torch.isnan(h), torch.isnan(rh)) and torch.equal(h.nan_to_num(0.5), rh.nan_to_num(0.5))
    if y is not None:
        ok = torch.isfinite(ry).all(dim=1)
        i8ref.check_y(y[ok], ry[ok], i8ref.RSTD_TOL * ry[ok].abs(), "y")
    if codes is not None:
        assert torch.equal(codes, rc), f"{int((codes != rc).sum())} codes differ"
        i8ref.check_scale(scale, rs, "scale")


NORM_SHAPES = [(1, 16), (1, 4096), (2, 8192), (3, 64), (5, 80), (7, 272), (33, 1040), (64, 2048), (65, 5008), (130, 256),
               (9, 16384), (3, 20000), (2, 65536), (700, 4096), (4100, 512), (3000, 128)]


@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm_matches_the_definition(M, K):
    _check_norm(_rows(M, K, 1), _rows(M, K, 2), (1 + 0.2 * _rows(1, K, 3, 0.0)[0].float()).to(BF16))


@pytest.mark.parametrize("r", [False, True])
@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("outs", [(True, True, True), (True, False, True), (False, True, True), (False, True, False),
                                  (True, True, False), (False, False, True)])
def test_norm_with_every_choice_of_arguments(r, w, outs):
    M, K = 37, 1168
    _check_norm(_rows(M, K, 4), _rows(M, K, 5) if r else None, _rows(1, K, 6, 0.0)[0] if w else None,
                h=outs[0], y=outs[1], codes=outs[2])


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("M,K", [(3, 64), (50, 2048), (20, 16384)])
def test_norm_in_place(which, M, K):
    _check_norm(_rows(M, K, 7), _rows(M, K, 8), _rows(1, K, 9, 0.0)[0], in_place=which)


def _special_rows(K):
    """Zero, tiny, huge, subnormal, outlier, constant rows; one value alone;
    alternating signs; squares that overflow and underflow binary32."""
    x = torch.zeros(12, K)
    g = torch.Generator().manual_seed(11)
    n = torch.randn(K, generator=g)
    x[1] = n * 1e-30
    x[2] = n * 1e30
    x[3] = n * 2.0 ** -130
    x[4] = n
    x[4, K // 2] = 3e4
    x[5] = -1.0
    x[6, K - 1] = 0.5
    x[7] = torch.where(torch.arange(K) % 2 == 0, 1.0, -1.0)
    x[8] = n * 1e-20
    x[9] = n * 1e36
    x[10] = n * 2.0 ** -70
    x[11, 0] = -3e38
    return x.to(BF16)


@pytest.mark.parametrize("K", [16, 512, 4096, 16400])
def test_rows_of_every_magnitude(K):
    x = _special_rows(K)
    _check_norm(x, None, None, eps=1e-6)
    _check_norm(x, None, None, eps=1e-30)
    _check_norm(x, torch.zeros_like(x), torch.ones(K, dtype=BF16))
    _check_quant(x)


@pytest.mark.parametrize("K", [16, 512, 4096, 16400])
def test_gains_of_every_magnitude(K):
    """Products that leave binary32 in rows that do not."""
    x = _special_rows(K)
    one = 1 + 0.2 * _rows(1, K, 42, 0.0)[0].float()
    for e in (-133, -120, -60, 60, 110):
        w = (one * 2.0 ** e).to(BF16)
        _check_norm(x, None, w)
        _check_norm(x, torch.zeros_like(x), w, eps=1e-30)
    w = (one.clamp(-1.9, 1.9) * 2.0 ** 127).to(BF16)  # y overflows, the scales do not
    assert torch.isfinite(i8ref.rmsnorm(x, None, w, 1e-6)[3].float()).all()
    _check_norm(x, None, w, y=False)
    w[::2] *= 2.0 ** -126
    w[1::4] = 0.0
    _check_norm(x, x, w, y=False)


@pytest.mark.parametrize("n,K", [(350, 4096), (345, 4240), (180, 8176), (176, 8192), (110, 12304), (100, 16384)])
def test_many_long_rows(n, K):
    """Each of n * 12 rows as the same row among twelve."""
    x = torch.cat([_special_rows(K)[1:], _rows(1, K, 40)])
    w = (1 + 0.2 * _rows(1, K, 41, 0.0)[0].float()).to(BF16)
    _, ry, rc, rs = i8ref.rmsnorm(x, None, w, 1e-6)
    for r in (None, torch.zeros_like(x)):
        xs, rs_ = x.repeat(n, 1), None if r is None else r.repeat(n, 1)
        _, y, codes, scale = (t if t is None else t.view(n, 12, *t.shape[1:]) for t in _norm(xs, rs_, w))
        i8ref.check_y(y[0], ry, i8ref.RSTD_TOL * ry.abs(), "y")
        i8ref.check_scale(scale[0], rs, "scale")
        assert torch.equal(codes[0], rc)
        for t in (y, codes, scale):
            assert torch.equal(t, t[:1].expand_as(t))


@pytest.mark.parametrize("K", [16, 4096])
def test_rows_with_nan_or_infinity_are_marked(K):
    x = _rows(6, K, 12)
    x[1, 3] = math.nan
    x[2, K - 1] = math.inf
    x[4, 0] = -math.inf
    _check_norm(x, None, None, y=False)
    _check_norm(x, _rows(6, K, 13), _rows(1, K, 14, 0.0)[0], y=False)
    _check_quant(x)
    w = torch.ones(K, dtype=BF16)
    w[5] = math.inf  # 0 * inf in a row of zeros, inf in the others
    x = _rows(3, K, 15)
    x[1] = 0.0
    _check_norm(x, None, w, y=False)


def _check_quant(x):
    M, K = x.shape
    codes = torch.full((M + 1, K), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((M + 1,), 7.0, device="cuda")
    ll.ll_quantize_i8(x.cuda(), M, K, codes[:M], scale[:M])
    torch.cuda.synchronize()
    assert torch.all(codes[M] == 77) and scale[M] == 7.0
    rc, a = i8ref.codes_of(x)
    assert torch.equal(codes[:M].cpu(), rc)
    # one division: the correctly rounded quotient
    want = (a.float() / 127.0)
    assert torch.equal(torch.nan_to_num(scale[:M].cpu(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))


@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_quantize_matches_the_definition(M, K):
    _check_quant(_rows(M, K, 16))


def test_codes_at_and_beside_every_border():
    """Values on the borders between codes (127 u / a = n + 1/2 for a = 254 *
    2^-j) and one bf16 step to each side, for every code and sign; and with a
    gain, products with 16 significant bits next to a border."""
    n = torch.arange(0, 127, dtype=torch.float64)
    tie = (2 * n + 1)  # with a = 254: 127 u / a = u / 2
    vals = tie.float().to(BF16)
    step = lambda t, d: (t.view(torch.int16) + d).view(BF16)  # noqa: E731
    u = torch.cat([vals, step(vals, 1), step(vals, -1), vals[:3]])
    K = (len(u) + 16) // 16 * 16
    x = torch.zeros(4, K, dtype=BF16)
    x[0, : len(u)] = u
    x[1, : len(u)] = -u
    x[2, : len(u)] = u * 2.0 ** -20
    x[3, : len(u)] = u * 2.0 ** 90
    x[0, -1], x[1, -1], x[2, -1], x[3, -1] = 254.0, 254.0, -254.0 * 2.0 ** -20, 254.0 * 2.0 ** 90
    _check_quant(x)
    # Products h * w * 2^-j of 16 significant bits below a, the ones whose
    # quotient is nearest to a border: ties, and quotients that one binary32
    # multiplication by 127 / a puts on the wrong side.
    K = 2048
    i = torch.arange(128, 256, dtype=torch.float64)
    p = (i[:, None] * i)[:, :, None] * 2.0 ** -torch.arange(0, 9, dtype=torch.float64)
    for h0, w0 in ((255.0, 254.0), (254.0, 252.0), (254.0, 241.0)):
        a = h0 * w0
        off = torch.where(p <= a, ((127.0 * p / a) % 1.0 - 0.5).abs(), torch.ones_like(p)).reshape(-1)
        near = torch.argsort(off)[: K - 1]
        h, w = torch.full((2, K), h0), torch.full((K,), w0)
        h[0, 1:], w[1:] = (i[near // (128 * 9)] * 2.0 ** -(near % 9)).float(), i[near // 9 % 128].float()
        h[1] = torch.where(torch.arange(K) % 2 == 1, -h[0], h[0])
        plain = torch.round((h * w) * (torch.tensor(127.0) / torch.tensor(a, dtype=torch.float32)))
        assert (plain != i8ref.codes_of(h.double() * w.double())[0]).sum() >= 20
        _check_norm(h.to(BF16), None, w.to(BF16))


@pytest.mark.parametrize("on_side_stream", [False, True])
def test_norm_and_quantize_are_captured_and_replayed(on_side_stream):
    M, K = 40, 2048
    x, r, w = _rows(M, K, 18).cuda(), _rows(M, K, 19).cuda(), _rows(1, K, 20, 0.0)[0].cuda()
    h, y = torch.empty_like(x), torch.empty_like(x)
    c, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        ll.ll_rmsnorm_i8(x, r, w, 1e-6, M, K, h, y, c, s)
    x2 = _rows(M, K, 21)
    x.copy_(x2)
    torch.cuda.synchronize()
    if on_side_stream:
        with torch.cuda.stream(st):
            g.replay()
    else:
        g.replay()
    torch.cuda.synchronize()
    rh, _, rc, rs = i8ref.rmsnorm(x2, r.cpu(), w.cpu(), 1e-6)
    assert torch.equal(h.cpu(), rh) and torch.equal(c.cpu(), rc)
    i8ref.check_scale(s, rs)


# ------------------------------------------------------------------ product
def _product_inputs(M, K, N, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    xs = torch.rand(M, generator=g) * 0.03 + 0.01
    ws = (torch.rand(N, generator=g) - 0.3) / (70.0 * math.sqrt(K))
    b = (torch.randn(N, generator=g) * 0.5).to(BF16) if bias else None
    return xq, xs, wq, ws, b


def _layer(wq, ws, b, gelu=False):
    layer = ll.Int8LinearLayer(wq.shape[0], wq.shape[1], ll.LL_EPILOGUE_GELU_TANH if gelu else ll.LL_EPILOGUE_NONE)
    layer.set_weights(wq.cuda(), ws.cuda(), None if b is None else b.cuda())
    return layer


def _forward(layer, xq, xs, stream=None):
    M = xq.shape[0]
    out = torch.full((M + 1, layer.N), 7.0, dtype=BF16, device="cuda")
    layer.forward(xq.cuda(), xs.cuda(), out=out[:M], stream=stream)
    torch.cuda.synchronize()
    assert ll.ll_i8_status(layer.handle) == ll.LL_OK
    assert torch.all(out[M] == 7.0), "a row behind the last was written"
    return out[:M]


def _check_product(M, K, N, bias=True, gelu=False, seed=30):
    xq, xs, wq, ws, b = _product_inputs(M, K, N, seed, bias)
    layer = _layer(wq, ws, b, gelu)
    y = _forward(layer, xq, xs)
    ref, size = i8ref.product(xq, xs, wq, ws, b, gelu)
    i8ref.check_y(y, ref, i8ref.PRODUCT_TOL * size, f"{M} x {K} -> {N}")
    assert torch.equal(_forward(layer, xq, xs), y)  # and the same again
    layer.close()


PRODUCT_SHAPES = [(1, 16, 8), (1, 4096, 1000), (2, 64, 136), (3, 2048, 2048), (4, 1040, 24), (5, 128, 128),
                  (8, 8192, 256), (15, 272, 520), (16, 4096, 4096), (17, 144, 3000), (31, 512, 64), (33, 1000 * 16, 8),
                  (48, 640, 1032), (64, 4096, 2048), (65, 2000, 136), (100, 1040, 1000), (127, 256, 264),
                  (128, 2048, 512), (129, 2064, 128), (200, 4096, 1024), (255, 80, 256), (256, 1024, 2048),
                  (257, 272, 504), (333, 1040, 1000), (384, 4096, 768), (511, 128, 2056), (512, 2048, 2048),
                  (700, 336, 120), (1025, 512, 1536), (1300, 2048, 2048), (2500, 144, 4096),
                  # features on the pairs' long side, tokens in narrow tiles
                  (65, 2064, 16384), (96, 4096, 16392), (128, 4096, 16384), (257, 1024, 16392), (300, 4096, 16384),
                  (80, 2048, 8192), (129, 2064, 8200), (257, 1040, 18944),
                  # streaming without a split of K, and one K step
                  (40, 4096, 16392), (7, 64, 2048), (200, 16, 8), (64, 128, 19000)]


@pytest.mark.parametrize("M,K,N", PRODUCT_SHAPES)
def test_product_matches_the_definition(M, K, N):
    _check_product(M, K, N, bias=(M + N) % 3 != 0, gelu=False, seed=M + K + N)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 512, 264), (30, 2048, 384), (150, 272, 136), (600, 512, 1000),
                                   (33, 256, 19000), (300, 4096, 16384)])
def test_product_with_gelu(M, K, N, bias):
    _check_product(M, K, N, bias=bias, gelu=True, seed=M)


@pytest.mark.parametrize("M", [1, 20, 200, 500])
def test_largest_sums_stay_exact(M):
    """Codes of -128 on both sides over the longest reduction: the sum is one
    product below 2^31; and alternating signs, which cancel to a small sum."""
    K, N = 131056, 16
    xq = torch.full((M, K), -128, dtype=torch.int8)
    wq = torch.full((N, K), -128, dtype=torch.int8)
    wq[1] = 127
    wq[2, ::2] = 127
    wq[3, 5:] = 0
    xs, ws = torch.full((M,), 2.0 ** -20), torch.ones(N)
    y = _forward(_layer(wq, ws, None), xq, xs)
    ref, size = i8ref.product(xq, xs, wq, ws, None, False)
    i8ref.check_y(y, ref, i8ref.PRODUCT_TOL * size)
    # size bounds the rounding of the exact sum: the cancelled sums are exact too
    assert torch.all((y.cpu().double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_a_nan_scale_gives_a_row_of_nan_and_touches_no_other(M):
    xq, xs, wq, ws, b = _product_inputs(M, 528, 200, 31)
    layer = _layer(wq, ws, b)
    want = _forward(layer, xq, xs).cpu()
    xs2 = xs.clone()
    xs2[M // 2] = math.nan
    y = _forward(layer, xq, xs2).cpu()
    assert torch.isnan(y[M // 2]).all()
    keep = torch.arange(M) != M // 2
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("M", [2, 100, 300, 700])
def test_scales_far_from_one(M):
    """Scales whose product leaves binary32 although every output is in range,
    and sums of zero under scales whose product is infinite."""
    xq, xs, wq, ws, _ = _product_inputs(M, 256, 520, 34)
    xq[0] = 0
    xs = torch.where(torch.arange(M) % 2 == 0, 1e30, 1e-25) * (xs + 1)
    ws = torch.where(torch.arange(520) % 2 == 0, 1e25, 1e-30) * (ws.abs() + 1)
    y = _forward(_layer(wq, ws, None), xq, xs).cpu()
    ref, size = i8ref.product(xq, xs, wq, ws, None, False)
    seen = (ref.abs() < 1e38) & ((ref == 0) | (ref.abs() > 1e-35))
    assert seen.float().mean() > 0.4 and torch.all(y[0] == 0)
    i8ref.check_y(y[seen], ref[seen], i8ref.PRODUCT_TOL * size[seen])


def test_layer_refusals():
    xq, xs, wq, ws, b = (t.cuda() for t in _product_inputs(4, 64, 16, 32))
    layer = ll.Int8LinearLayer(16, 64)
    y = torch.empty(4, 16, dtype=BF16, device="cuda")

    def code(fn):
        with pytest.raises(ll.LLError) as e:
            fn()
        return e.value.code

    assert code(lambda: layer.forward(xq, xs, out=y)) == ll.LL_ERR_NOT_READY
    bad = ws.clone()
    bad[3] = math.inf
    assert code(lambda: layer.set_weights(wq, bad, b)) == ll.LL_ERR_INVALID_ARG
    assert code(lambda: layer.set_weights(wq.cpu(), ws, b)) == ll.LL_ERR_INVALID_ARG
    assert code(lambda: layer.set_weights(wq[:, :32], ws, b)) == ll.LL_ERR_INVALID_ARG
    layer.set_weights(wq, ws, b)
    want = layer.forward(xq, xs)
    for fn in (lambda: layer.forward(xq, xs, out=y.float()), lambda: layer.forward(xq.t(), xs),
               lambda: layer.forward(xq, xs[:2]), lambda: layer.forward(xq.float(), xs),
               lambda: ll.ll_i8_forward(layer.handle, xq, xs, y, -1),
               lambda: ll.ll_i8_forward(layer.handle, xq.cpu(), xs, y, 4),
               lambda: ll.ll_i8_forward(layer.handle, xq, xs.cpu(), y, 4),
               lambda: ll.ll_i8_forward(layer.handle, xq, xs, y.cpu(), 4),
               lambda: ll.ll_i8_forward(layer.handle, xq, xs, xq, 4),
               lambda: ll.ll_i8_forward(layer.handle, xq.data_ptr() + 8, xs, y, 4),
               lambda: layer.set_weights(wq, bad, None)):
        assert code(fn) == ll.LL_ERR_INVALID_ARG
    assert code(lambda: ll.ll_i8_set_epilogue(layer.handle, ll.LL_EPILOGUE_GEGLU_TANH)) == ll.LL_ERR_UNSUPPORTED
    assert code(lambda: ll.ll_i8_set_epilogue(layer.handle, 9)) == ll.LL_ERR_INVALID_ARG
    ll.ll_i8_forward(layer.handle, xq, xs, y, 0)
    assert torch.equal(layer.forward(xq, xs), want)  # refused calls changed nothing


@pytest.mark.parametrize("M,N", [(1, 264), (40, 2048), (200, 136), (600, 520), (3000, 2048)])
def test_withheld_loads_time_out_and_the_layer_recovers(M, N):
    """Every device-side wait is bounded: with loads withheld the waits run
    out, the status tells so and is cleared, and the layer works again."""
    xq, xs, wq, ws, b = _product_inputs(M, 1040, N, 33)
    layer = _layer(wq, ws, b)
    want = _forward(layer, xq, xs)
    x, s = xq.cuda(), xs.cuda()
    ll.ll_i8_set_debug(layer.handle, True, 1_000_000)
    layer.forward(x, s)
    torch.cuda.synchronize()
    assert ll.ll_i8_status(layer.handle) == ll.LL_ERR_DEVICE_TIMEOUT
    assert ll.ll_i8_status(layer.handle) == ll.LL_OK
    ll.ll_i8_set_debug(layer.handle, False, 2_000_000_000)
    assert torch.equal(_forward(layer, xq, xs), want)
    ref, size = i8ref.product(xq, xs, wq, ws, b, False)
    i8ref.check_y(want, ref, i8ref.PRODUCT_TOL * size)


def test_two_layers_and_two_streams_at_once():
    """Forwards of one layer on two streams, another layer beside them, and a
    captured graph of each replayed at the same time."""
    ins = [_product_inputs(M, 2048, 1024, 40 + M) for M in (24, 300)]
    layer = _layer(*ins[0][2:5])
    other = _layer(*ins[1][2:5], gelu=True)
    dev = [(i[0].cuda(), i[1].cuda()) for i in ins]
    outs = [torch.zeros(d[0].shape[0], 1024, dtype=BF16, device="cuda") for d in dev for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def go():
        for rep in range(20):
            for k, (c, s) in enumerate(dev):
                layer.forward(c, s, out=outs[2 * k], stream=streams[k])
                other.forward(c, s, out=outs[2 * k + 1], stream=streams[1 - k])

    go()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for k in range(2):
        for j, (l, gelu) in enumerate(((0, False), (1, True))):
            ref, size = i8ref.product(ins[k][0], ins[k][1], *ins[l][2:5], gelu)
            i8ref.check_y(got[2 * k + j], ref, i8ref.PRODUCT_TOL * size)
    graphs = []
    for k, (c, s) in enumerate(dev):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[k]):
            layer.forward(c, s, out=outs[2 * k])
            other.forward(c, s, out=outs[2 * k + 1])
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for rep in range(20):
        for k, g in enumerate(graphs):
            with torch.cuda.stream(streams[k]):
                g.replay()
    torch.cuda.synchronize()
    assert ll.ll_i8_status(layer.handle) == ll.LL_OK and ll.ll_i8_status(other.handle) == ll.LL_OK
    for a, b in zip(outs, got):
        assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in x, the codes, the weight and y: the first and
    the last rows."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(70)
    M, K = 65600, 32768
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    for part in (x[:3], x[-3:]):
        part.copy_(torch.randn(3, K, generator=g, device="cuda"))
    codes, scale = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    ll.ll_quantize_i8(x, M, K, codes, scale)
    h, y = torch.empty_like(x), torch.empty_like(x)
    nc, ns = torch.empty_like(codes), torch.empty_like(scale)
    ll.ll_rmsnorm_i8(x, x, None, 1e-6, M, K, h, y, nc, ns)
    for rows in (slice(0, 4), slice(M - 4, M)):
        xc = x[rows].cpu()
        rc, a = i8ref.codes_of(xc)
        assert torch.equal(codes[rows].cpu(), rc) and torch.equal(scale[rows].cpu(), a.float() / 127.0)
        rh, ry, rc, rs = i8ref.rmsnorm(xc, xc, None, 1e-6)
        assert torch.equal(h[rows].cpu(), rh) and torch.equal(nc[rows].cpu(), rc)
        i8ref.check_y(y[rows], ry, i8ref.RSTD_TOL * ry.abs())
        i8ref.check_scale(ns[rows], rs)
    del x, codes, h, y, nc
    # y of 2.3e9 elements
    M, K, N = 140000, 64, 16392
    xq, xs, wq, ws, b = _product_inputs(M, K, N, 71)
    out = torch.empty(M, N, dtype=BF16, device="cuda")
    _layer(wq, ws, b).forward(xq.cuda(), xs.cuda(), out=out)
    for rows in (slice(0, 5), slice(M - 5, M)):
        ref, size = i8ref.product(xq[rows], xs[rows], wq, ws, b, False)
        i8ref.check_y(out[rows], ref, i8ref.PRODUCT_TOL * size)
    del out
    # a weight of 2.2e9 codes, on both kernels that stream it
    N, K = 16904, 130000
    wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    ws = torch.rand(N, generator=g, device="cuda") * 1e-5
    layer = ll.Int8LinearLayer(N, K)
    layer.set_weights(wq, ws)
    for M in (3, 300):
        xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8, device="cuda")
        xs = torch.rand(M, generator=g, device="cuda")
        got = layer.forward(xq, xs)
        for cols in (slice(0, 9), slice(N - 9, N)):
            ref, size = i8ref.product(xq.cpu(), xs.cpu(), wq[cols].cpu(), ws[cols].cpu(), None, False)
            i8ref.check_y(got[:, cols], ref, i8ref.PRODUCT_TOL * size)
    assert ll.ll_i8_status(layer.handle) == ll.LL_OK


def test_empty_batches():
    x, c, s = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 64, dtype=torch.int8, device="cuda"), \
        torch.empty(0, device="cuda")
    ll.ll_rmsnorm_i8(x, x, None, 1e-6, 0, 64, x, x, c, s)
    ll.ll_quantize_i8(x, 0, 64, c, s)
    layer = _layer(*_product_inputs(1, 64, 24, 74)[2:])
    assert layer.forward(c, s).shape == (0, 24)
    assert layer.forward(c.view(0, 5, 64), s.view(0, 5)).shape == (0, 5, 24)
    with pytest.raises(ll.LLError) as e:  # and the other end: refused before any address is looked at
        ll.ll_i8_forward(layer.handle, None, None, None, 2 ** 31 - 511)
    assert e.value.code == ll.LL_ERR_UNSUPPORTED


def test_tensors_of_other_strides_are_refused():
    """Column slices, transposes, expanded rows: the library takes an address
    only, so the binding refuses what is not contiguous."""
    x = _rows(8, 128, 72).cuda()
    c, s = torch.empty(8, 64, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    for bad in (x[:, :64], x[:, ::2], x.t()[:8], x[:1, :64].expand(8, 64), x[:, :64].float(), x[:, :64].cpu()):
        with pytest.raises(ll.LLError) as e:
            ll.ll_quantize_i8(bad, 8, 64, c, s)
        assert e.value.code == ll.LL_ERR_INVALID_ARG
    with pytest.raises(ll.LLError) as e:
        ll.ll_rmsnorm_i8(x, None, x[:, 0], 1e-6, 8, 128, None, torch.empty_like(x), None, None)
    assert e.value.code == ll.LL_ERR_INVALID_ARG
    # leading dimensions may be split: batch x sequence
    layer = _layer(*_product_inputs(1, 128, 24, 73)[2:])
    c, s = torch.empty(2, 4, 128, dtype=torch.int8, device="cuda"), torch.empty(2, 4, device="cuda")
    ll.ll_quantize_i8(x.view(2, 4, 128), 8, 128, c, s)
    y = layer.forward(c, s)
    assert y.shape == (2, 4, 24)
    assert torch.equal(y.view(8, 24), layer.forward(c.view(8, 128), s.view(8)))
    # a row slice is contiguous, and its address need only be 16-byte aligned
    odd = torch.empty(8 * 128 + 8, dtype=BF16, device="cuda")[8:].view(8, 128)
    odd.copy_(x)
    c, s = torch.empty(8, 128, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")[1:]
    ll.ll_quantize_i8(odd, 8, 128, c, s)
    assert torch.equal(c.cpu(), i8ref.codes_of(x.cpu())[0])


# ------------------------------------------------------------------- chain
def _block(M, K, F, seed):
    """Buffers and layers of a feed-forward, and its step: the residual stream
    in `h` takes the block's output."""
    g = torch.Generator().manual_seed(seed)
    up = ll.Int8LinearLayer.from_dense((torch.randn(F, K, generator=g) / math.sqrt(K)).to(BF16).cuda(),
                                       epilogue=ll.LL_EPILOGUE_GELU_TANH)
    down = ll.Int8LinearLayer.from_dense((torch.randn(K, F, generator=g) / math.sqrt(F)).to(BF16).cuda())
    t = dict(h=_rows(M, K, seed).cuda(), d=_rows(M, K, seed + 1).cuda(), w=_rows(1, K, seed + 2, 0.0)[0].cuda(),
             c1=torch.empty(M, K, dtype=torch.int8, device="cuda"), s1=torch.empty(M, device="cuda"),
             mid=torch.empty(M, F, dtype=BF16, device="cuda"),
             c2=torch.empty(M, F, dtype=torch.int8, device="cuda"), s2=torch.empty(M, device="cuda"))

    def step(wait=lambda: None):
        ll.ll_rmsnorm_i8(t["d"], t["h"], t["w"], 1e-6, M, K, t["h"], None, t["c1"], t["s1"])
        wait()
        up.forward(t["c1"], t["s1"], out=t["mid"])
        wait()
        ll.ll_quantize_i8(t["mid"], M, F, t["c2"], t["s2"])
        wait()
        down.forward(t["c2"], t["s2"], out=t["d"])
        wait()

    return t, step


@pytest.mark.parametrize("M", [1, 48, 200, 700])
def test_back_to_back_steps_equal_steps_one_by_one(M):
    """Every kernel may start before the one ahead of it has ended, and each
    step overwrites buffers that the step before still reads: 30 steps without a
    wait, the same 30 captured in one graph, and 30 with a wait after every
    call give the same bits."""
    results = []
    for mode in range(3):
        t, step = _block(M, 512, 1536, 80)
        torch.cuda.synchronize()
        if mode == 0:
            for _ in range(30):
                step(torch.cuda.synchronize)
        elif mode == 1:
            for _ in range(30):
                step()
        else:
            h0, d0 = t["h"].clone(), t["d"].clone()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for _ in range(30):
                    step()
            t["h"].copy_(h0)
            t["d"].copy_(d0)
            g.replay()
        torch.cuda.synchronize()
        results.append((t["h"].cpu(), t["d"].cpu()))
    for r in results[1:]:
        assert torch.equal(r[0], results[0][0]) and torch.equal(r[1], results[0][1])
    assert torch.isfinite(results[0][0].float()).all()


@pytest.mark.parametrize("M", [1, 40, 333])
def test_feed_forward_of_norm_product_quantisation_product(M):
    """The operators as a feed-forward uses them: residual + norm -> codes,
    int8 product with GELU, quantisation, int8 product.  Each step is checked
    against its definition applied to the values that it was given."""
    K, F = 512, 2048
    g = torch.Generator().manual_seed(50 + M)
    x, r, w = _rows(M, K, 51), _rows(M, K, 52), _rows(1, K, 53, 0.0)[0]
    W1 = (torch.randn(F, K, generator=g) / math.sqrt(K)).to(BF16)
    W2 = (torch.randn(K, F, generator=g) / math.sqrt(F)).to(BF16)
    b1 = (0.1 * torch.randn(F, generator=g)).to(BF16)
    up = ll.Int8LinearLayer.from_dense(W1.cuda(), b1.cuda(), ll.LL_EPILOGUE_GELU_TANH)
    down = ll.Int8LinearLayer.from_dense(W2.cuda())
    h = torch.empty(M, K, dtype=BF16, device="cuda")
    c1, s1 = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    c2, s2 = torch.empty(M, F, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    ll.ll_rmsnorm_i8(x.cuda(), r.cuda(), w.cuda(), 1e-6, M, K, h, None, c1, s1)
    mid = up.forward(c1, s1)
    ll.ll_quantize_i8(mid, M, F, c2, s2)
    y = down.forward(c2, s2)
    torch.cuda.synchronize()
    rh, _, rc, rs = i8ref.rmsnorm(x, r, w, 1e-6)
    assert torch.equal(h.cpu(), rh) and torch.equal(c1.cpu(), rc)
    i8ref.check_scale(s1, rs)
    wc1, wa1 = i8ref.codes_of(W1)
    wc2, wa2 = i8ref.codes_of(W2)
    ref, size = i8ref.product(c1.cpu(), s1.cpu(), wc1, (wa1.float() / 127.0), b1, True)
    i8ref.check_y(mid, ref, i8ref.PRODUCT_TOL * size)
    rc2, a2 = i8ref.codes_of(mid.cpu())
    assert torch.equal(c2.cpu(), rc2) and torch.equal(s2.cpu(), a2.float() / 127.0)
    ref, size = i8ref.product(c2.cpu(), s2.cpu(), wc2, (wa2.float() / 127.0), None, False)
    i8ref.check_y(y, ref, i8ref.PRODUCT_TOL * size)
    # And the whole against the unquantised block.  A quantised row is off by
    # max / rms / (127 sqrt(12)) of its norm: 17 / 440 for the norm's rows
    # (loud channels), 10 / 440 for the GELU's, 5 / 440 for each weight; times
    # GELU's slope of at most 1.13: under 0.1 even if all of them add up.
    u = i8ref.rmsnorm(x, r, w, 1e-6)[1]
    full = i8ref.gelu_tanh(u @ W1.double().t() + b1.double()) @ W2.double().t()
    off = (y.cpu().double() - full).norm() / full.norm()
    assert off < 0.1, float(off)


def test_norm_output_feeds_a_lite_linear_layer():
    """The bf16 output of the norm is the input of the low-rank + FP8 layer."""
    from llgpu import check
    import oracle
    from synth_inputs import make_inputs, to_numpy_bits
    inp = make_inputs(70, 512, 264, 16, seed=60)
    w = _rows(1, 512, 61, 0.0)[0]
    y = torch.empty(70, 512, dtype=BF16, device="cuda")
    ll.ll_rmsnorm_i8(inp.x.cuda(), None, w.cuda(), 1e-6, 70, 512, None, y, None, None)
    layer = ll.LiteLinearLayer(264, 512, 16, inp.scale_mode)
    layer.set_weights(inp.A.cuda(), inp.B.cuda(), inp.Q.cuda(), inp.scale.cuda(), inp.bias.cuda())
    out = layer.forward(y)
    torch.cuda.synchronize()
    bits = [to_numpy_bits(t) for t in (y.cpu(), inp.B, inp.A, inp.Q, inp.scale)]
    check(out.cpu(), oracle.forward(*bits, inp.scale_mode, to_numpy_bits(inp.bias)), what="norm into layer")
    layer.close()
