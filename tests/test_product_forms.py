"""Which form of the product the shapes of the GPU tests take (CPU): every form runs there, in both
activations and with replica slots, however the choice is tuned."""

import pytest

from tests.product_shapes import SHAPES
from tests.rules import FORMS, form


@pytest.mark.parametrize("shape", SHAPES)
def test_the_shapes_take_the_forms_that_they_name(shape):
    rows, R, E, S, N, D, plain, swiglu = shape
    n_inst = R * (E // R + S)
    assert form(rows, n_inst, N, D, False) == plain
    assert form(rows, n_inst, N // 2, D, True) == swiglu


def test_every_form_has_a_shape_with_slots():
    assert {s[6] for s in SHAPES if s[3]} == set(FORMS)
    # a block of 16 channels cannot hold gates and their ups
    assert {s[7] for s in SHAPES if s[3]} == set(FORMS) - {"16x16"}
