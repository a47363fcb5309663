"""Sampling and norm where their rules and number formats end."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from test_gpu_norm_mx import FMT, dev, host, strided  # noqa: E402
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

# ---- norm ----------------------------------------------------------------------------

@pytest.mark.parametrize("form", ["fp8", "fp4"])
@pytest.mark.parametrize("d", [256, 4096])
@pytest.mark.parametrize("off", [0, 1])
def test_norm_of_tiny_weights_is_rounded_once(off, d, form):
    """y below float32's normal numbers, whose float32 lies half between two codes far more often: every code is that of y
    itself, in rows of any alignment.  (y in 64 bits is off by 2^-50, and no y comes so near to a tie.)"""
    rng = np.random.default_rng([d, len(form)])
    x = rng.standard_normal((1 << 20) // d * d).reshape(-1, d).astype(np.float32)
    w = (rng.uniform(1, 2, d) * 2.0 ** -rng.integers(125, 140, d // 32).repeat(32)).astype(np.float32)
    mx = pb.empty_mx(len(x), d, FMT[form])
    pb.pi_rms_norm(pb.make_norm(dev(w)), strided(x, 0, 0.0, off)[0], mx=mx)
    torch.cuda.synchronize()
    y = R.norm(x, w, 1e-5)
    codes, want = host(mx._keep[0]), R.packed(R.codes(y, form), form)
    assert np.array_equal(host(mx._keep[1]), R.scales(y, form))
    assert int((codes != want).sum()) == 0


@pytest.mark.parametrize("tokens,heads,token_stride,head_stride", [(5, 4, 1, 5), (5, 4, 4, 1), (3, 3, 2, 3), (2, 3, 7, 2), (4, 2, 2, 5)])
def test_norm_writes_rows_in_any_order(tokens, heads, token_stride, head_stride):
    """Rows that lie between each other without meeting, and what lies between them."""
    d = 64
    rng = np.random.default_rng(tokens)
    x = rng.standard_normal((tokens, heads, d)).astype(np.float32)
    flat = torch.full((40 * d,), 7.0, device="cuda")
    y = flat.as_strided((tokens, heads, d), (token_stride * d, head_stride * d, 1))
    pb.pi_rms_norm(pb.make_norm(None, d=d), dev(x), y=y)
    torch.cuda.synchronize()
    want = R.norm(x, None, 1e-5)
    assert (np.abs(host(y) - want) <= 2.0 ** -22 * np.abs(want)).all()
    places = {i * token_stride + j * head_stride for i in range(tokens) for j in range(heads)}
    assert len(places) == tokens * heads
    assert all(bool((flat[p * d:(p + 1) * d] == 7).all()) for p in range(40) if p not in places)


# places of x and y in rows of ten heads: first head, and heads from one to the next
@pytest.mark.parametrize("x_at,y_at", [((0, 1), (3, 1)), ((0, 1), (7, 1)), ((1, 2), (0, 2)), ((0, 2), (5, 2)), ((0, 3), (8, 1)),
                                       ((4, 1), (0, 2))])
def test_norm_between_the_rows_of_its_input(x_at, y_at):
    """Heads of a fused row normed into other heads of the same rows."""
    tokens, heads, d = 6, 3, 64
    if y_at == (8, 1) or x_at == (4, 1):
        heads = 2
    rng = np.random.default_rng(x_at)
    before = rng.standard_normal((tokens, 10, d)).astype(np.float16)
    fused = dev(before)
    x, y = (fused[:, at:at + (heads - 1) * step + 1:step] for at, step in (x_at, y_at))
    want = R.norm(before[:, x_at[0]::x_at[1]][:, :heads], None, 1e-5)
    pb.pi_rms_norm(pb.make_norm(None, d=d), x, y=y)
    torch.cuda.synchronize()
    after = host(fused)
    places = [y_at[0] + i * y_at[1] for i in range(heads)]
    assert (np.abs(after[:, places] - want) <= 2.0 ** -10.9 * np.abs(want) + 2.0 ** -25).all()
    rest = [i for i in range(10) if i not in places]
    assert np.array_equal(after[:, rest], before[:, rest])


@pytest.mark.parametrize("off", [0, 1])
def test_norm_past_float32(off):
    """A y past float32's largest value is infinite in every output; its neighbours' blocks are as they are."""
    d = 128
    x = np.ones((3, d), np.float32)
    w = np.ones(d, np.float32)
    x[1, 40], w[40] = 50, 3e38
    y, mx = torch.empty((3, d), device="cuda"), pb.empty_mx(3, d, pb.PI_MXFP8)
    pb.pi_rms_norm(pb.make_norm(dev(w)), strided(x, 0, 0.0, off)[0], y=y, mx=mx)
    torch.cuda.synchronize()
    want = R.norm(x, w, 1e-5)
    assert want[1, 40] > 3.5e38 > want[0, 40]
    got = host(y)
    assert np.isinf(got[1, 40]) and np.isfinite(np.delete(got.reshape(-1), d + 40)).all()
    with np.errstate(over="ignore"):
        seen = want.astype(np.float32).astype(np.float64)
    assert np.array_equal(host(mx._keep[1]), R.scales(seen, "fp8"))
    assert list(host(mx._keep[1])[1]) == [R.scales(want[1:2], "fp8")[0, 0], 255, *R.scales(want[1:2], "fp8")[0, 2:]]
