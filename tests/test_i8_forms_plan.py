"""The cases of test_gpu_i8_forms run on the forms that they are named for."""
import pytest

import rank_fp8_residual_b200 as ll
import test_gpu_i8_forms as forms


@pytest.mark.parametrize("nk,form,M", forms.CASES)
def test_cases_are_planned_on_their_forms(nk, form, M):
    assert forms.form_of(*nk, M) == form


EVERY = {forms.SPLIT, forms.DIRECT, forms.STAGED, forms.PAIR, forms.SWAP}


def test_every_form_has_a_case():
    assert {form for _, form, _ in forms.CASES} == EVERY
    assert set(forms.REMAINDERS) == EVERY and set(forms.STEPS) == EVERY


@pytest.mark.parametrize("form", sorted(EVERY))
def test_remainders_and_steps_are_planned_on_their_forms(form):
    """And leave a part of a tile of tokens, of features and of the reduction."""
    for M, K, N in forms.REMAINDERS[form]:
        assert forms.form_of(N, K, M) == form
        _, features, tokens, _ = ll.ll_i8_plan(N, K, M, 148)
        assert M % tokens and N % features and K % 128
    M, K, F = forms.STEPS[form]
    assert forms.form_of(F, K, M) == form


@pytest.mark.parametrize("M,K,N,form", [
    # us, this form and the next best of another
    (100, 1024, 28000, forms.SWAP),  # 9.8, 11.5 streaming, 12.3 pairs
    (65, 1024, 28000, forms.SWAP),   # 9.1, 11.0 streaming
    (65, 2048, 8192, forms.SWAP),    # 7.3, 7.7 streaming
    (257, 4096, 8192, forms.SWAP),   # 12.7, 14.7 pairs
    (200, 1040, 18936, forms.PAIR), (640, 1024, 28000, forms.PAIR), (65, 4096, 8192, forms.SPLIT)])
def test_measured_crossovers_of_the_swapped_pairs(M, K, N, form):
    assert forms.form_of(N, K, M) == form
