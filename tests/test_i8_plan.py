"""Dispatch of the int8 layer (ll_i8_plan, host arithmetic) at the measured
crossovers on 148 SMs, and limits that hold for every plan."""
import random

import pytest

import rank_fp8_residual_b200 as ll
import test_gpu_i8

S, P, W = ll.LL_I8_STREAM, ll.LL_I8_PAIR, ll.LL_I8_PAIR_SWAP


# (M, K, N): what measured faster there
@pytest.mark.parametrize("M,K,N,kernel", [
    (1, 4096, 16384, S), (64, 4096, 16384, S), (256, 4096, 16384, P), (300, 4096, 16384, W), (512, 4096, 16384, P),
    (64, 4096, 4096, S), (128, 4096, 4096, S), (256, 4096, 4096, P), (32, 1024, 1024, S), (128, 1024, 1024, P),
    (96, 4096, 16384, S), (160, 4096, 16384, S), (200, 4096, 16384, P), (128, 1024, 16384, S), (128, 4096, 8192, W),
    (40, 4096, 19000, W), (64, 128, 19000, S), (64, 1024, 28000, S), (100, 4096, 19000, P), (256, 8192, 2048, S), (64, 2048, 2048, S), (3630, 2048, 8192, P), (16384, 4096, 16384, P)])
def test_measured_crossovers(M, K, N, kernel):
    assert ll.ll_i8_plan(N, K, M, 148)[0] == kernel


def test_streaming_splits_fill_the_gpu():
    assert ll.ll_i8_plan(16384, 4096, 1, 148) == (S, 128, 16, 1)  # 128 tiles
    assert ll.ll_i8_plan(4096, 4096, 1, 148) == (S, 128, 16, 4)   # 32 tiles x 4 CTAs
    assert ll.ll_i8_plan(2048, 2048, 20, 148) == (S, 128, 32, 8)
    assert ll.ll_i8_plan(8, 16, 1, 148) == (S, 128, 16, 1)        # one K step


def test_every_plan_is_within_the_kernels_limits():
    rng = random.Random(0)
    for _ in range(3000):
        M = int(2 ** rng.uniform(0, 15))
        N = 8 * int(2 ** rng.uniform(0, 12))
        K = 16 * int(2 ** rng.uniform(0, 12.9))
        kernel, tf, tt, splits = ll.ll_i8_plan(N, K, M, rng.choice([148, 132, 2, 74]))
        steps = (K + 127) // 128
        if kernel == S:
            assert M <= 256 and tf == 128 and tt % 16 == 0 and M <= tt < M + 16
            assert 1 <= splits <= min(8, steps)
        else:
            assert splits == 1
            wide, w = (tt, tf) if kernel == P else (tf, tt)
            assert wide == 256 and 64 <= w <= 256 and w % 32 == 0


@pytest.mark.parametrize("args", [(0, 64, 1, 148), (12, 64, 1, 148), (8, 8, 1, 148), (8, 64, 0, 148), (8, 64, 1, 1)])
def test_plan_refuses(args):
    with pytest.raises(ll.LLError) as e:
        ll.ll_i8_plan(*args)
    assert e.value.code == ll.LL_ERR_INVALID_ARG


def test_the_gpu_tests_reach_every_kernel():
    """The shapes of the GPU tests cover the three forms, split and unsplit
    streaming tiles and several tile widths."""
    plans = [ll.ll_i8_plan(N, K, M, 148) for M, K, N in test_gpu_i8.PRODUCT_SHAPES]
    assert {p[0] for p in plans} == {S, P, W}
    assert {p[3] > 1 for p in plans if p[0] == S} == {True, False}
    assert len({p[1] for p in plans if p[0] == P}) >= 4 and len({p[2] for p in plans if p[0] == W}) >= 2
