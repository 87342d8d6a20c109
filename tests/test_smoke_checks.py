"""The smoke step's comparison of the attention with the oracle: mistakes planted in the result are seen."""
import numpy as np
import pytest

import __graft_entry__ as entry
from oracle import attention as oa


def case():
    """A prompt whose first key's value is 0 in some places: error and bound are both 0 there."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((9, 4, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64))
    v[0, :, ::5] = 0.0
    want, _, spread, _ = oa.attend(q, k, v, 0.125)
    bound = 2.0 ** -8 * np.abs(want) + 1.05 * 2.0 ** -8 * spread
    assert (bound == 0).any()
    return want, bound


def test_a_right_result_passes():
    want, bound = case()
    got = want + 0.5 * bound
    assert 0.4 < entry._part_of_bound(got, want, bound, "prompt") < 0.6
    assert entry._part_of_bound(want, want, np.zeros_like(bound), "prompt") == 0.0


@pytest.mark.parametrize("wrong", [1000.0, float("nan"), float("inf")])
@pytest.mark.parametrize("everywhere", [True, False])
def test_a_wrong_result_does_not(wrong, everywhere):
    want, bound = case()
    got = want.copy()
    if everywhere:
        got[bound > 0] += wrong
    else:
        got[3, 1, 7] += wrong
    with pytest.raises(AssertionError, match="off by more"):
        entry._part_of_bound(got, want, bound, "prompt")


def test_a_wrong_zero_does_not():
    want, bound = case()
    got = want.copy()
    got[0, 0, 0] = 1e-30
    with pytest.raises(AssertionError, match="off by more"):
        entry._part_of_bound(got, want, bound, "prompt")
