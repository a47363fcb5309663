"""GPU parity of sampling against its definition in 64 bits (step_ref.py): the same token, count and probability."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run(logits, u, t=None, k=None, p=None, m=None, pad=0, off=0, stream=None):
    rows, vocab = logits.shape
    flat = torch.full((off + rows * (vocab + pad),), float("inf"), dtype=torch.from_numpy(logits).dtype, device=DEV)
    view = flat[off:].view(rows, vocab + pad)[:, :vocab]
    view.copy_(dev(logits))
    out = [torch.full((rows + 1,), -7, dtype=d, device=DEV) for d in (torch.int32, torch.float32, torch.int32)]
    ws = torch.full((pb.pi_sample_workspace_bytes(rows, vocab),), 255, dtype=torch.uint8, device=DEV)
    f32 = lambda v: dev(None if v is None else np.asarray(v, np.float32))  # noqa: E731
    rule = pb.make_sample_rule(f32(t), dev(None if k is None else np.asarray(k, np.int32)), f32(p), f32(m))
    pb.pi_sample(view, rule, f32(u), out[0], out[1], out[2], ws, stream)
    torch.cuda.synchronize()
    assert all(int(x[rows]) == -7 for x in out)
    return [x[:rows].cpu().numpy() for x in out]


def check(logits, u, t=None, k=None, p=None, m=None, **kw):
    """prob: a float32 rounding (2^-24) of a quotient of integers, each weight within 2^-44 of the first; where a choice
    came within 2^-36 of another outcome (2^20 weights off by 2^-44 at most, of a sum of at least 1, would be 2^-24; random
    ones add up to 2^-34 at their worst) the inputs are changed beforehand, not the check: no case below comes so near."""
    token, prob, kept = run(logits, u, t, k, p, m, **kw)
    at = lambda v, i: None if v is None else np.float32(v[i]) if v is not k else int(v[i])  # noqa: E731
    for i in range(len(logits)):
        want = R.sample(logits[i], np.float32(u[i]), at(t, i), at(k, i), at(p, i), at(m, i))
        assert want[3] > 2.0 ** -36, ("the inputs lie on a border", i, want)
        assert (token[i], kept[i]) == (want[0], want[2]), (i, token[i], kept[i], prob[i], want)
        assert abs(prob[i] - want[1]) <= 2.0 ** -23 * want[1] + 2.0 ** -40


def rows_of(rng, rows, vocab, dtype, sharp=2.0):
    x = sharp * rng.standard_normal((rows, vocab)) + 6.0 * (rng.random((rows, vocab)) < 0.001)
    return x.astype(np.float16 if dtype == "f16" else np.float32)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 63), (4, 64), (7, 1000), (3, 4097), (2, 50007), (2, 128000), (1, 200003)])
def test_rules(rows, vocab, dtype):
    rng = np.random.default_rng([rows, vocab])
    l = rows_of(rng, rows, vocab, dtype)
    u = rng.random(rows).astype(np.float32)
    t = rng.uniform(0.5, 1.5, rows).astype(np.float32)
    k = rng.integers(1, min(vocab, 200) + 1, rows).astype(np.int32)
    p, m = rng.uniform(0.3, 0.99, rows).astype(np.float32), rng.uniform(0.01, 0.3, rows).astype(np.float32)
    check(l, u)
    check(l, u, t)
    check(l, u, t, k)
    check(l, u, t, p=p, pad=3, off=1)
    check(l, u, m=m)
    check(l, u, t, k, p)
    check(l, u, t, k, p, m, pad=8)
    check(l, u, 0 * t)
    check(l, u, k=np.full(rows, vocab, np.int32))
    check(l, u, k=np.ones(rows, np.int32), pad=1)
    check(l, u, p=np.full(rows, 1e-9, np.float32))


def test_rows_with_rules_of_their_own():
    rng = np.random.default_rng(3)
    n = 60
    l = rows_of(rng, n, 5003, "f32")
    kind = np.arange(n) % 6
    t = np.where(kind == 0, 0, np.where(kind == 1, np.nan, rng.uniform(0.3, 2, n))).astype(np.float32)
    k = np.where(kind == 2, rng.integers(1, 3000, n), np.where(kind == 3, -5, 0)).astype(np.int32)
    p = np.where(kind == 4, rng.uniform(0.1, 0.999, n), np.where(kind == 3, np.nan, 1.5)).astype(np.float32)
    m = np.where(kind == 5, rng.uniform(0.001, 0.5, n), np.where(kind == 4, np.nan, -1)).astype(np.float32)
    check(l, rng.random(n).astype(np.float32), t, k, p, m)


@pytest.mark.parametrize("vocab", [70, 9000, 60000])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_equal_logits_go_by_index(dtype, vocab):
    """All tokens alike, and a few values that most tokens share: counts and sums end inside the ties."""
    rng = np.random.default_rng(vocab)
    n = 6
    few = rng.integers(-3, 3, (n, vocab)).astype(np.float16 if dtype == "f16" else np.float32)
    few[:, ::7] *= -1                                             # zeros of both signs
    u = rng.random(n).astype(np.float32)
    for l in (few, np.full_like(few, 2.5)):
        check(l, u, k=rng.integers(1, vocab, n).astype(np.int32))
        # (no sum of equal weights comes near these parts of the whole)
        check(l, u, p=np.array([0.1003, 0.3007, 0.5003, 0.7001, 0.9009, 0.9907], np.float32))
        check(l, u, k=np.full(n, vocab // 2 + 1, np.int32), p=np.array([0.1003, 0.3007, 0.5003, 0.7001, 0.9009, 0.9907], np.float32))
        check(l, u, m=np.full(n, 0.99, np.float32))
        check(l, u, np.zeros(n, np.float32))


def test_a_sum_that_reaches_top_p_exactly():
    """Equal weights are exact: of 4096 tokens the first 1024 reach a quarter, and no more are kept."""
    l = np.zeros((3, 4096), np.float32)
    token, prob, kept = run(l, [0.0, 0.5, 1.0], p=[0.25, 0.5, 1e-30])
    assert list(kept) == [1024, 2048, 1] and list(token) == [0, 1024, 0]
    assert np.array_equal(prob, np.array([2.0 ** -10, 2.0 ** -11, 1], np.float32))


def test_random_numbers_at_their_ends():
    l = np.log(np.array([[1, 2, 3, 2, 1e-30]] * 7)).astype(np.float32)
    u = np.array([0, -1, np.nan, 1, 2, np.inf, 1 - 2.0 ** -24], np.float32)
    token, _, _ = run(l, u)
    # (the last token's weight is none of the sum's 2^-43)
    assert list(token) == [0, 0, 0, 3, 3, 3, 3]


@pytest.mark.parametrize("vocab", [50, 20011])
def test_infinities_and_nan(vocab):
    rng = np.random.default_rng(1)
    l = rows_of(rng, 9, vocab, "f32")
    l[0] = -np.inf
    l[1] = np.nan
    l[2, ::2], l[2, 1::2] = np.nan, -np.inf
    l[3, rng.random(vocab) < 0.5] = -np.inf
    l[4, rng.random(vocab) < 0.5] = np.nan
    l[5] = -np.inf
    l[5, vocab - 1] = -3e38                                       # a mask of the type's lowest values beside one
    l[6, [3, 40]] = np.inf
    l[7] = np.finfo(np.float32).min
    l[8] = np.where(rng.random(vocab) < 0.9, np.finfo(np.float32).min, l[8])
    u = rng.random(9).astype(np.float32)
    ks = [None, np.full(9, 5, np.int32), np.full(9, vocab, np.int32)]
    for k in ks:
        for p in (None, np.full(9, 0.7003, np.float32)):
            for m in (None, np.full(9, 0.05, np.float32)):
                check(l, u, k=k, p=p, m=m)
    check(l, u, np.zeros(9, np.float32))
    check(l, u, np.full(9, 1e-30, np.float32))
    check(l, u, np.full(9, 1e30, np.float32), k=np.full(9, 5, np.int32))


@pytest.mark.parametrize("temperature", [1e-3, 50.0, 1e4, np.inf])
def test_sharp_and_flat(temperature):
    """One token that takes all, and distributions in which all weigh nearly or exactly alike."""
    rng = np.random.default_rng(8)
    l = rows_of(rng, 4, 30011, "f32", 3.0)
    t, u = np.full(4, temperature, np.float32), rng.random(4).astype(np.float32)
    check(l, u, t)
    check(l, u, t, k=np.array([1, 100, 9000, 30000], np.int32))
    check(l, u, t, p=np.array([0.1003, 0.3007, 0.9001, 0.9993], np.float32))
    check(l, u, t, k=np.full(4, 20000, np.int32), p=np.array([0.1003, 0.3007, 0.9001, 0.9993], np.float32))


def test_top_k_below_the_weights_that_count():
    """The k-th token weighs nothing any more: counts stay exact."""
    rng = np.random.default_rng(2)
    l = np.linspace(0, -4000, 9001, dtype=np.float32)[None, rng.permutation(9001)].repeat(3, 0)
    l[1, rng.permutation(9001)[:3000]] = -1e9                     # an outlier far below the others
    check(l, [0.1, 0.6, 0.99], k=[4000, 7000, 9000])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_borders_in_long_rows(dtype):
    """Rows of many chunks whose borders lie where many tokens are: top-k and top-p far down, alone and together, ties at them."""
    rng = np.random.default_rng(12)
    l = rows_of(rng, 8, 70001, dtype, 1.0)
    l[6:] = np.round(l[6:] * 4) / 4                               # a few values, thousands of tokens each
    u = rng.random(8).astype(np.float32)
    k = np.array([1, 2, 5000, 30000, 69000, 70001, 20000, 60000], np.int32)
    p = np.array([0.0103, 0.3007, 0.5003, 0.9007, 0.9993, 0.99993, 0.4003, 0.8507], np.float32)
    t = np.array([0.2, 1, 3, 1, 0.7, 1, 1, 2], np.float32)
    check(l, u, t, k=k)
    check(l, u, t, p=p)
    check(l, u, t, k=k, p=p)
    check(l, u, t, k=k, p=p, m=np.full(8, 0.01, np.float32), pad=5, off=3)
    check(l, u, t, k=np.full(8, 40, np.int32), p=p)


def test_calls_on_two_streams_and_after_each_other():
    """The same workspace for one call after another, others for calls at the same time: every call as it is alone."""
    rng = np.random.default_rng(4)
    l = [dev(rows_of(rng, n, v, "f32")) for n, v in ((3, 90001), (17, 5000))]
    u = [dev(rng.random(x.shape[0]).astype(np.float32)) for x in l]
    rule = [pb.make_sample_rule(top_k=torch.full((x.shape[0],), 40, dtype=torch.int32, device=DEV),
                                top_p=torch.full((x.shape[0],), 0.9, device=DEV)) for x in l]
    ws = [torch.full((pb.pi_sample_workspace_bytes(*x.shape),), 255, dtype=torch.uint8, device=DEV) for x in l]
    alone = []
    for x, r, n, w in zip(l, rule, u, ws):
        token, prob = torch.empty(x.shape[0], dtype=torch.int32, device=DEV), torch.empty(x.shape[0], device=DEV)
        pb.pi_sample(x, r, n, token, prob, None, w)
        torch.cuda.synchronize()
        alone.append((token.clone(), prob.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[(torch.empty_like(t), torch.empty_like(p)) for _ in range(10)] for t, p in alone]
    torch.cuda.synchronize()
    for i in range(10):
        for x, r, n, w, s, o in zip(l, rule, u, ws, streams, outs):
            pb.pi_sample(x, r, n, o[i][0], o[i][1], None, w, stream=s)
    torch.cuda.synchronize()
    for (t, p), o in zip(alone, outs):
        assert all(torch.equal(a, t) and torch.equal(b, p) for a, b in o)


def test_draws_follow_the_distribution():
    """20000 rows of one distribution, evenly spaced numbers: each token as often as its weight says, within one row."""
    l = np.array([[0.0, 1.0, -np.inf, 2.0, 1.5, -1.0]], np.float32)
    n = 20000
    token, _, _ = run(np.repeat(l, n, 0), (np.arange(n) + 0.5) / n)
    w = np.exp(l[0].astype(np.float64))
    assert (np.abs(np.bincount(token, minlength=6) - n * w / w.sum()) <= 1.0).all()


def test_wrong_tensors():
    l, u, tok = torch.zeros((2, 10), device=DEV), torch.zeros(2, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    ws = torch.empty(pb.pi_sample_workspace_bytes(2, 10), dtype=torch.uint8, device=DEV)
    for kw in (dict(u=torch.zeros(1, device=DEV)), dict(token=tok.long()), dict(logits=torch.zeros((10, 2), device=DEV).t()),
               dict(rule=pb.make_sample_rule(temperature=torch.ones(1, device=DEV))), dict(u=torch.zeros(2))):
        a = dict(logits=l, rule=pb.make_sample_rule(), u=u, token=tok) | kw
        with pytest.raises(ValueError):
            pb.pi_sample(a["logits"], a["rule"], a["u"], a["token"], ws=ws)
    with pytest.raises(pb.PiError):
        pb.pi_sample(l, pb.make_sample_rule(), u, tok, ws=ws[:0])


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("vocab", [1, 1000, 4096, 4097, 8191, 8192])
def test_short_rows_and_long_rows_agree(vocab, dtype):
    """A row alone, among 300, and with tokens that are never kept behind it: the same bits.  Equal logits are among them."""
    rng = np.random.default_rng([vocab, 5])
    rows = 300
    l = rows_of(rng, rows, vocab, dtype)
    l[::7] = np.round(l[::7])
    l[::50], l[3::50, ::2] = 1.0, -np.inf
    u = rng.random(rows).astype(np.float32)
    t = np.where(np.arange(rows) % 5, rng.uniform(0.3, 2, rows), 0).astype(np.float32)
    k, p = rng.integers(-5, 300, rows).astype(np.int32), rng.uniform(0.2, 1.2, rows).astype(np.float32)
    padded = np.concatenate([l, np.full((rows, 8300 - vocab), -np.inf, l.dtype)], 1)
    for rules in (dict(t=t), dict(t=t, k=k), dict(t=t, p=p), dict(t=t, k=k, p=p, m=0.1 * p)):
        many = run(l, u, **rules)
        for lo, hi in ((0, 100), (100, 101), (101, 300)):
            few = run(l[lo:hi], u[lo:hi], **{name: v[lo:hi] for name, v in rules.items()})
            assert all(np.array_equal(a, b[lo:hi]) for a, b in zip(few, many)), (lo, hi)
        assert all(np.array_equal(a, b) for a, b in zip(run(padded, u, **rules), many))
        assert all(np.array_equal(a, b[:200]) for a, b in zip(run(padded[:200], u[:200], **{n: v[:200] for n, v in rules.items()}), many))
