"""Sampling and norm where their rules and number formats end."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_sample import run as draw  # noqa: E402

pytestmark = pytest.mark.gpu


# ---- sampling ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("vocab", [70, 9000, 60000])
def test_min_p_above_one_keeps_the_first_alone(vocab, dtype):
    """No weight reaches a min-p above 1, so the first token alone is kept, however many are as large; at 1 all of these."""
    rng = np.random.default_rng(vocab)
    l = rng.integers(-3, 3, (6, vocab)).astype(dtype)
    l[2, ::5] = np.inf
    l[3, ::2] = np.nan
    l[4] = 1.5                                                    # (more than a list holds, where the row is long)
    l[5] = -np.inf
    ok = np.where(np.isnan(l), -np.inf, l)
    best = ok.max(1)
    first, many = ok.argmax(1), (ok == best[:, None]).sum(1)
    assert (many[:5] > 1).all()
    u = np.full(6, 0.9, np.float32)
    some = np.full(6, max(2, vocab // 3), np.int32)
    for more in (dict(), dict(k=some), dict(p=np.full(6, 0.7, np.float32)), dict(k=some, p=np.full(6, 0.7, np.float32)),
                 dict(t=np.full(6, 1e30, np.float32))):
        for m in (np.nextafter(np.float32(1), np.float32(2)), np.float32(1.5), np.float32(np.inf)):
            token, prob, kept = draw(l, u, m=np.full(6, m, np.float32), **more)
            assert list(token) == [*first[:5], -1] and list(kept) == [1] * 5 + [0]
            assert list(prob) == [1.0] * 5 + [0.0]
    _, prob, kept = draw(l, u, m=np.ones(6, np.float32))
    assert list(kept) == [*many[:5], 0]
    assert np.array_equal(prob[:5], (1 / many[:5]).astype(np.float32))
