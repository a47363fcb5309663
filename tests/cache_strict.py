"""Comparison of attention outputs with the definition that no NaN passes: where one
side holds a NaN or an infinity, the other has to hold the same."""
import numpy as np

import cache_ref as R


def compare(got, got_lse, r, f16):
    """got and got_lse (float64) against r of cache_ref.attention; rows of no sequence hold 7."""
    tol, tol_lse = R.attention_tolerance(r, f16)
    mine = r["mine"]
    assert (got[~mine] == 7.0).all() and (got_lse[~mine] == 7.0).all(), "a row of no sequence was written"
    empty = mine & (r["seen"] == 0)
    assert (got[empty] == 0).all() and np.isneginf(got_lse[empty]).all(), "a row that sees nothing"
    m = mine & ~empty
    for name, a, b, t in (("out", got[m], r["out"][m], tol[m]), ("lse", got_lse[m], r["lse"][m], tol_lse[m])):
        assert np.array_equal(np.isnan(a), np.isnan(b)), f"{name}: NaN in other places"
        inf = np.isinf(a) | np.isinf(b)
        assert np.array_equal(a[inf], b[inf]), f"{name}: infinities in other places"
        fine = np.isfinite(b)
        err = np.abs(a[fine] - b[fine])
        assert (err <= t[fine]).all(), f"{name}: {(~(err <= t[fine])).sum()} of {err.size} off"


def check(case, got, got_lse, **rule):
    """test_gpu_cache.Case.check, strictly."""
    with np.errstate(all="ignore"):
        r = R.attention(case.q, case.k[case.layer], case.v[case.layer], case.table, case.q_start, case.lens,
                        float(np.float32(case.scale)), **rule)
        compare(got, got_lse, r, case.dtype == "f16")
