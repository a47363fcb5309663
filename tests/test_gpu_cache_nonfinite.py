"""Infinities and NaN in what a row sees, and rules at the ends of 32 bits: the result does not depend on how
the keys are shared out over waves and splits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_ref as R  # noqa: E402
import cache_strict  # noqa: E402
import test_gpu_cache as G  # noqa: E402

pytestmark = pytest.mark.gpu

# query heads, key heads, new tokens, lengths: one short sequence, waves with and without keys, a split over the keys,
# tiles of many rows, such tiles split, f32 tiles of few rows beside them
SHAPES = [(2, 1, [1], [1]), (2, 1, [1], [70]), (4, 2, [1, 2], [700, 300]), (8, 1, [1], [9001]), (2, 1, [100], [300]),
          (2, 1, [70], [5000]), (2, 1, [1, 130, 3], [700, 140, 300])]


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(G.Case, "check", cache_strict.check)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
def test_nan_queries(dtype, hq, hk, new, lens):
    """A row with a NaN query gets NaN, not what a row that sees nothing gets; the others nothing of it."""
    c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=20)
    c.q[-1, 0, 5] = np.nan
    if c.T > 1:
        c.q[0, -1] = np.nan
    c.run()
    c.run(cap=10.0)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
@pytest.mark.parametrize("sharp", [1.0, 60.0])
def test_nan_keys(dtype, hq, hk, new, lens, sharp):
    """One NaN key, wherever it lies, reaches every row that sees it: also from a wave or a split whose other scores
    weigh nothing (sharp), or that has no other keys."""
    for at in (0, 0.3, 0.5, 0.77, 1):
        c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=21, sharp=sharp)
        for s, n in enumerate(lens):
            c.k[0][c.place(s, int(at * (n - 1)))] = np.nan
        c.run()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
def test_nan_in_every_key(dtype, hq, hk, new, lens):
    c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=22)
    c.k[..., 3] = np.nan
    c.run()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
@pytest.mark.parametrize("plant", [np.nan, np.inf])
def test_values_that_weigh_nothing(dtype, hq, hk, new, lens, plant):
    """A NaN or an infinity in V at a key whose score is far below the others' stays in the row's output, also where
    the keys around it (all that a wave has, perhaps) are as low."""
    for at in (0, 0.3, 0.5, 0.77, 1):
        for around in (1, 32, 256):
            c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=23, sharp=0.1)
            c.q[..., 0] = 60.0
            c.k[..., 0] = 30.0
            for s, n in enumerate(lens):
                key = int(at * (n - 1))
                for j in range(key // around * around, min(key // around * around + around, n)):
                    p = c.place(s, j)
                    c.k[0, p[0], :, p[2], 0] = -30.0           # 450 below the others, in natural units
                p = c.place(s, key)
                c.v[0, p[0], :, p[2], 7] = plant
            got, _ = c.run(check=False)
            for t, s, pos in R.positions(c.q_start, c.lens):
                sees = pos >= int(at * (lens[s] - 1))
                assert np.isfinite(got[t, :, 7]).all() != sees and np.isfinite(got[t, :, :7]).all(), (t, pos, at)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
@pytest.mark.parametrize("plant", [1.0, np.nan, np.inf])
def test_scores_of_minus_infinity_alone(dtype, hq, hk, new, lens, plant):
    """A row whose scores are all -inf gets zeros and lse = -inf, whatever V holds."""
    c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=24)
    c.q[..., 0] = 1.0
    c.k[..., 0] = -np.inf
    c.v[:] = plant
    got, lse = c.run(check=False)
    assert (got == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
@pytest.mark.parametrize("scale", [3e38, -3e38, 1e-45])
def test_scales_at_the_ends_of_32_bits(dtype, hq, hk, new, lens, scale):
    """Scores of 0 stay 0: a plain mean."""
    c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=25)
    c.scale = scale
    c.q[:] = 0
    c.run()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
def test_a_bias_at_the_end_of_32_bits(dtype, hq, hk, new, lens):
    """A slope so steep that a row attends to its own key alone, whose distance is 0."""
    c = G.Case(dtype, hq, hk, 64, 16, new, lens, seed=26)
    c.run(slopes=np.full(hq, 3e38))


@pytest.mark.parametrize("hq,hk,new,lens", SHAPES)
def test_large_values_at_keys_that_weigh_nothing(hq, hk, new, lens):
    """f32 values of 10^36 at keys far below the last ones leave nothing in the output."""
    c = G.Case("f32", hq, hk, 64, 16, new, lens, seed=27, sharp=0.1)
    c.q[..., 0] = 60.0
    c.k[..., 0] = 30.0
    for s, n in enumerate(lens):
        far = -(-n // 3)
        for j in range(far):
            p = c.place(s, j)
            c.k[0, p[0], :, p[2], 0] = -30.0
            if n > 3:
                c.v[0, p[0], :, p[2]] *= 1e36
    c.run()
