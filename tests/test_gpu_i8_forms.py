"""The int8 layer on every form of its kernels: split streaming, unsplit
streaming (straight stores and staged ones), CTA pairs in both orientations.
The cases name the form that they are meant for, and test_i8_forms_plan checks
that they are planned so."""
import pytest
import torch

import rank_fp8_residual_b200 as ll
from test_gpu_i8 import _forward, _layer, _product_inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# (N, K) of a layer -> tokens per form
SPLIT, DIRECT, STAGED, PAIR, SWAP = "split", "direct", "staged", "pair", "swap"
NARROW = (2056, 2064)
WIDE = (16392, 4096)
FORMS = {NARROW: {SPLIT: 20, PAIR: 300}, WIDE: {DIRECT: 5, STAGED: 40, SWAP: 300, PAIR: 512}}
CASES = [(nk, form, M) for nk, forms in FORMS.items() for form, M in forms.items()]


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
