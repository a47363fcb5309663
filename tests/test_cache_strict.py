"""The strict comparison rejects what it should: planted mistakes in the expected outputs, on the CPU."""
import numpy as np
import pytest

import cache_ref as R
from cache_strict import compare


@pytest.fixture
def case():
    rng = np.random.default_rng(0)
    k, v = (rng.standard_normal((4, 1, 8, 16)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((5, 2, 16)).astype(np.float16)
    v[1, 0, 7] = np.nan                                     # key 15: the last row sees it
    with np.errstate(all="ignore"):
        r = R.attention(q, k, v, np.array([[0, 1], [-1, -1]]), np.array([0, 4, 5]), np.array([16, 4]), 0.25)
    return r, r["out"].copy(), r["lse"].copy()


def test_the_definition_passes(case):
    r, out, lse = case
    assert np.isnan(out[3]).all() and np.isfinite(out[:3]).all() and (out[4] == 0).all()
    compare(out, lse, r, True)


@pytest.mark.parametrize("plant", [np.nan, np.inf, -np.inf, 100.0])
@pytest.mark.parametrize("where", ["out", "lse"])
@pytest.mark.parametrize("row", [0, 4])
def test_a_planted_value_is_found(case, plant, where, row):
    r, out, lse = case
    (out if where == "out" else lse)[row] = plant
    if where == "lse" and row == 4 and plant == -np.inf:
        return compare(out, lse, r, True)                   # what a row that sees nothing holds
    with pytest.raises(AssertionError):
        compare(out, lse, r, True)


def test_a_lost_nan_and_an_output_of_nothing_but_nan_are_found(case):
    r, out, lse = case
    lost = out.copy()
    lost[3] = 0
    for bad in (lost, np.full_like(out, np.nan)):
        with pytest.raises(AssertionError):
            compare(bad, lse, r, True)
