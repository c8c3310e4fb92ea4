"""TreeVerifier's settings, as far as they need no GPU."""
import numpy as np
import pytest

import tree_speculative_decoding_04_b200 as tv
from tree_speculative_decoding_04_b200.verifier import TreeVerifier, _layer_windows


@pytest.mark.parametrize("window", [7, np.int64(7), np.int32(7), np.uint16(7), [7, 7, 7], np.array([7, 7, 7])])
def test_a_window_is_any_integer_or_one_for_each_layer(window):
    got = _layer_windows(window, 3)
    assert got == [7, 7, 7] and all(type(w) is int for w in got)


def test_a_window_for_each_layer_must_match_the_layers():
    with pytest.raises(tv.TVError, match="window: 2 entries for 3 layers"):
        _layer_windows([7, 0], 3)


@pytest.mark.parametrize("kw", [dict(softcap=-30.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
                                dict(window=-1), dict(window=[0, -4])])
def test_scores_that_would_be_left_out_are_refused(kw):
    with pytest.raises(tv.TVError, match=next(iter(kw))):
        TreeVerifier(1, 3, 4, 2, 64, 100, 2, 64, 3, device="cpu", **kw)
