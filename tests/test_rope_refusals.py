"""Numbers that are none in the arguments of rope_frequencies: refused, whichever they are."""
import math

import pytest

import kv_chunk_selection_b200 as lsa

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [dict(base=NAN), dict(base=INF), dict(factor=NAN), dict(factor=INF), dict(original_context=NAN),
                                 dict(original_context=-1), dict(slow=NAN), dict(fast=NAN)])
def test_parts_refuse(bad):
    args = dict(scaling="parts", factor=2.0, original_context=4096)
    lsa.rope_frequencies(64, **args)
    with pytest.raises(ValueError):
        lsa.rope_frequencies(64, **{**args, **bad})


def test_infinite_bounds_stay_what_the_formula_makes_of_them():
    plain, linear = lsa.rope_frequencies(64)[0], lsa.rope_frequencies(64, scaling="linear", factor=2.0)[0]
    assert (lsa.rope_frequencies(64, scaling="parts", factor=2.0, original_context=math.inf)[0] == plain).all()
    assert (lsa.rope_frequencies(64, scaling="parts", factor=2.0, original_context=4096, fast=math.inf)[0] == linear).all()
