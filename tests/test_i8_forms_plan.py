"""The cases of test_gpu_i8_forms run on the forms that they are named for."""
import pytest

import test_gpu_i8_forms as forms


@pytest.mark.parametrize("nk,form,M", forms.CASES)
def test_cases_are_planned_on_their_forms(nk, form, M):
    assert forms.form_of(*nk, M) == form


def test_every_form_has_a_case():
    assert {form for _, form, _ in forms.CASES} == {forms.SPLIT, forms.DIRECT, forms.STAGED, forms.PAIR, forms.SWAP}
