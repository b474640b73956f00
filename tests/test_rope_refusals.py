"""Numbers that are none in the arguments of rope_frequencies: refused, whichever they are."""
import pytest

import kv_chunk_selection_b200 as lsa

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad", [dict(base=NAN), dict(base=INF), dict(factor=NAN), dict(factor=INF), dict(original_context=NAN),
                                 dict(original_context=INF), dict(original_context=-1), dict(slow=NAN), dict(fast=NAN),
                                 dict(fast=INF)])
def test_parts_refuse(bad):
    args = dict(scaling="parts", factor=2.0, original_context=4096)
    lsa.rope_frequencies(64, **args)
    with pytest.raises(ValueError):
        lsa.rope_frequencies(64, **{**args, **bad})
