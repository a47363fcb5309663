"""GPU parity of the paged cache: attention over it, rotary positions with the
append, and the pages' bookkeeping, against the definitions in 64 bits
(cache_ref.py).  Tolerances follow from the stated roundings."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f16": torch.float16, "f32": torch.float32}


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


class Case:
    """Random cache, tables and queries: `new` tokens of every sequence over `lens`."""

    def __init__(self, dtype, hq, hk, d, page, new, lens, seed=0, layers=1, layer=0, spare=3, sharp=1.0, extra=1):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.hq, self.hk, self.d, self.page, self.layer = rng, dtype, hq, hk, d, page, layer
        self.new, self.lens = list(new), np.array(lens, dtype=np.int32)
        need = [-(-int(x) // page) for x in lens]
        self.pages = sum(need) + spare
        ids = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(need + [0]) + extra), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:]
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.q_start[-1])
        n16 = np.float16 if dtype == "f16" else np.float32
        self.k = rng.standard_normal((layers, self.pages, hk, page, d)).astype(n16)
        self.v = rng.standard_normal((layers, self.pages, hk, page, d)).astype(n16)
        self.q = (sharp * rng.standard_normal((self.T, hq, d))).astype(n16)
        self.scale = 1.0 / np.sqrt(d)

    def place(self, s, j):
        return self.table[s, j // self.page], slice(None), j % self.page

    def run(self, cap=0.0, slopes=None, window=0, prefix=None, first=None, stride=0, stream=None, check=True,
            max_new=None, max_len=None):
        k, v = dev(self.k, DT[self.dtype]), dev(self.v, DT[self.dtype])
        # queries as a slice of a wider product, the output with room between rows
        wide = torch.full((self.T, self.hq + stride, self.d), float("nan"), dtype=DT[self.dtype], device=DEV)
        wide[:, :self.hq] = dev(self.q, DT[self.dtype])
        out = torch.full((self.T, self.hq + stride, self.d), 7.0, dtype=DT[self.dtype], device=DEV)
        lse = torch.full((self.T, self.hq), 7.0, dtype=torch.float32, device=DEV)
        cache = pb.make_kv_cache(k, v)
        batch = pb.make_seq_batch(dev(self.q_start), dev(self.lens), dev(self.table), self.T,
                                  max(self.new + [0]) if max_new is None else max_new,
                                  int(self.lens.max()) if max_len is None else max_len)
        rule = pb.make_score_rule(self.scale, cap, None if slopes is None else dev(slopes, torch.float32), window,
                                  None if prefix is None else dev(prefix), None if first is None else dev(first))
        ws = torch.full((pb.pi_attention_workspace_bytes(cache, batch, self.hq),), 255, dtype=torch.uint8, device=DEV)
        q, o = wide[:, :self.hq], out[:, :self.hq]
        pb.pi_paged_attention(cache, self.layer, batch, rule, q, o, lse, ws, stream)
        torch.cuda.synchronize()
        assert (out[:, self.hq:] == 7.0).all()
        got, got_lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        if check:
            self.check(got, got_lse, cap=cap, slopes=slopes, window=window, prefix=prefix, first=first)
        return got, got_lse

    def check(self, got, got_lse, **rule):
        r = R.attention(self.q, self.k[self.layer], self.v[self.layer], self.table, self.q_start, self.lens,
                        float(np.float32(self.scale)), **rule)
        tol, tol_lse = R.attention_tolerance(r, self.dtype == "f16")
        mine = r["mine"]
        assert (got[~mine] == 7.0).all() and (got_lse[~mine] == 7.0).all()
        empty = mine & (r["seen"] == 0)
        assert (got[empty] == 0).all() and np.isneginf(got_lse[empty]).all()
        m = mine & ~empty
        fine = np.isfinite(r["out"][m])
        assert np.isnan(r["out"][m]).sum() == 0 or np.array_equal(np.isnan(got[m]), np.isnan(r["out"][m]))
        err = np.abs(np.where(fine, got[m], 0) - np.where(fine, r["out"][m], 0))
        bad = err > np.where(fine, tol[m], np.inf)
        assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(err / np.where(fine, tol[m], np.inf)):.2f} of the tolerance"
        inf = np.isinf(r["out"][m])
        assert np.array_equal(got[m][inf], r["out"][m][inf])
        ok = np.isfinite(r["lse"][m])
        assert (np.abs(got_lse[m][ok] - r["lse"][m][ok]) <= tol_lse[m][ok]).all()


def slopes(h):
    return 2.0 ** (-8.0 * (np.arange(h) + 1) / h)


# ---- attention -------------------------------------------------------------------

SHAPES = [  # query heads, key heads, head size, page
    (1, 1, 8, 8), (4, 4, 64, 16), (8, 1, 64, 32), (16, 2, 128, 16), (6, 2, 80, 16), (5, 5, 96, 8), (3, 1, 256, 64),
    (24, 1, 40, 128), (2, 2, 136, 16)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES)
def test_attention_single_tokens(dtype, hq, hk, d, page):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 515]
    Case(dtype, hq, hk, d, page, [1] * len(lens), lens, seed=d, sharp=2.0).run(stride=hk)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,d,page", SHAPES)
def test_attention_chunks(dtype, hq, hk, d, page):
    new, lens = [1, 3, 17, 40, 70, 0, 129], [1, 5, 17, 333, 200, 9, 150]
    Case(dtype, hq, hk, d, page, new, lens, seed=d + 1).run(stride=2)


RULES = {
    "cap": dict(cap=5.0), "bias": dict(bias=True), "window": dict(window=33), "window1": dict(window=1),
    "first": dict(first=37), "prefix": dict(prefix=[3, 90, 150, 1000]), "all": dict(cap=20.0, bias=True, window=70, first=50,
                                                                                   prefix=[3, 90, 170, 10])}


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rule", sorted(RULES))
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [2, 150, 33, 64]])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_rules(dtype, rule, new, d):
    c = Case(dtype, 8, 2, d, 16, new, [2, 333, 170, 64], seed=5, sharp=2.0)
    r = dict(RULES[rule])
    if r.pop("bias", False):
        r["slopes"] = slopes(8)
    if "prefix" in r:
        r["prefix"] = np.array(r["prefix"])
    if "first" in r:
        pos = np.array([p for _, _, p in R.positions(c.q_start, c.lens)])
        r["first"] = pos // r["first"] * r["first"]
    c.run(**r)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1, 1], [4, 5, 70, 3, 200]])
def test_attention_rows_that_see_nothing(dtype, new):
    """Lengths of zero, fewer keys than new tokens, a first key after the row, a window's start past a prefix."""
    c = Case(dtype, 4, 2, 64, 16, new, [0, 3, 65, 1, 300], seed=2)
    pos = np.array([p for _, _, p in R.positions(c.q_start, c.lens)])
    first = np.where(np.arange(c.T) % 3 == 0, pos + 1, np.where(np.arange(c.T) % 3 == 1, -5, 2 ** 31 - 1))
    c.run(first=first)
    c.run()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 70, 9]])
def test_attention_extreme_bounds(dtype, new):
    """Windows, prefixes and first keys at the ends of 32 bits, for rows before position 0 too."""
    c = Case(dtype, 4, 2, 64, 16, new, [20, 200, 3], seed=15)
    top = 2 ** 31 - 1
    for window in (top, 1, 0):
        for prefix in ([top, 10, 2], [-top - 1, -5, 1]):
            first = np.array([(-top - 1, 0, 5, top)[t % 4] for t in range(c.T)])
            c.run(window=window, prefix=np.array(prefix))
            c.run(window=window, prefix=np.array(prefix), first=first)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scale,cap", [(0.125, 30.0), (0.125, 2.0), (-0.125, 3.0), (0.02, 0.04), (1e-7, 1.0), (0.125, 1e6),
                                       (2e-6, 0.3), (0.0, 5.0), (50.0, 1.0)])
def test_attention_caps(scale, cap, bias):
    """Scores far under the cap, around half of it and past it, in one tile and apart; scales of any size."""
    c = Case("f16", 4, 2, 64, 16, [1, 70, 40], [90, 300, 140], seed=16)
    c.scale = scale
    c.q[::3] *= 0.25
    c.k[0][c.place(1, 100)] = 3.0
    c.run(cap=cap, slopes=slopes(4) if bias else None)


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 64), (4, 4, 80), (1, 1, 256)])
def test_attention_f32_tiles_of_few_rows(hq, hk, d):
    """Sequences of one to sixteen rows beside long ones, and a long one's last rows, with each rule and masked junk."""
    c = Case("f32", hq, hk, d, 16, [1, 130, 5, 0, 136, 8, 1], [700, 140, 5, 7, 500, 300, 33], seed=17)
    c.table[0, 20] = -1
    for s, j in ((0, 699), (1, 139), (4, 499)):
        c.v[0][c.place(s, j)] = np.nan
    first = np.array([max(0, p - 200) for _, _, p in R.positions(c.q_start, c.lens)])
    last = np.array([i for i, (_, s, p) in enumerate(R.positions(c.q_start, c.lens)) if p == c.lens[s] - 1])
    c.q[last] *= 2
    with np.errstate(all="ignore"):
        c.run(first=first)
        c.run(window=40)
        c.run(slopes=slopes(hq), cap=4.0)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("d", [64, 80, 128, 256])
def test_attention_masked_values_have_no_influence(dtype, new, d):
    """NaN and infinities in free pages, past a sequence's end and at keys that a row does not see."""
    c = Case(dtype, 4, 2, d, 16, [new, new], [135, 200], seed=3)
    c.k[:, c.free], c.v[:, c.free] = np.nan, np.inf
    for s in range(2):
        last, used = c.table[s, (int(c.lens[s]) - 1) // 16], int(c.lens[s]) % 16
        if used:
            c.k[0, last, :, used:], c.v[0, last, :, used:] = np.nan, -np.inf
    first = np.full(c.T, 20, dtype=np.int32)                     # keys before 20 are seen by no row
    for s in range(2):
        for j in range(20):
            p = c.place(s, j)
            c.k[0][p], c.v[0][p] = np.inf, np.nan
    c.run(first=first)
    if new > 1:                                                  # later tokens must not reach earlier rows
        for s in range(2):
            for j, x in ((int(c.lens[s]) - 1, np.nan), (int(c.lens[s]) - 40, np.inf), (int(c.lens[s]) - 70, -np.inf)):
                c.v[0][c.place(s, j)] = x
        with np.errstate(all="ignore"):
            c.run(first=first)
        for s in range(2):
            c.k[0][c.place(s, int(c.lens[s]) - 33)] = np.nan
        got, _ = c.run(first=first, check=False)
        for t, s, pos in R.positions(c.q_start, c.lens):
            if pos >= c.lens[s] - 33:
                assert np.isnan(got[t]).all()
            elif pos < c.lens[s] - 70:
                assert np.isfinite(got[t]).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("new", [1, 50])
def test_attention_entries_that_name_no_page(dtype, new):
    c = Case(dtype, 4, 2, 64, 16, [new, new], [300, 90], seed=4)
    c.table[0, 2], c.table[0, 7], c.table[1, 0], c.table[0, 11] = -1, c.pages, 2 ** 31 - 1, -2 ** 31
    c.run()


def test_attention_untrusted_counts():
    """Lengths past the table are cut to it, rows of no sequence are left alone."""
    c = Case("f16", 4, 2, 64, 16, [3, 2], [40, 33], seed=6, extra=0)
    c.lens[0] = 48                       # its three pages are full
    want, _ = c.run()
    c.lens[0] = 2 ** 31 - 1
    got, _ = c.run(check=False, max_len=48)
    assert np.array_equal(got[:3], want[:3])
    c = Case("f16", 4, 2, 64, 16, [3, 2], [40, 33], seed=6)
    c.q_start = np.array([1, 3, 4], dtype=np.int32)       # rows 0 and 4 belong to nobody
    c.run(max_new=2)
    c.lens[:] = -7
    c.run(max_new=2, max_len=0)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,d,new,length", [(8, 1, 128, 1, 9001), (2, 2, 64, 1, 20000), (4, 2, 128, 6, 7000), (2, 1, 64, 100, 5000)])
def test_attention_long(dtype, hq, hk, d, new, length):
    """Work split over the keys, and joined; twice the same bits."""
    c = Case(dtype, hq, hk, d, 32, [new], [length], seed=7, sharp=2.0)
    a = c.run()
    b = c.run(check=False)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("dtype,new", [("f16", [1] * 5), ("f16", [3, 40, 1, 90, 7]), ("f32", [1] * 5), ("f32", [3, 40, 1, 90, 7])])
def test_attention_bounds_are_hints(dtype, new):
    """max_len says nothing about the result, only about the split of the work."""
    c = Case(dtype, 4, 2, 64, 16, new, [700, 41, 3000, 95, 8], seed=8)
    for max_len in (0, 10, 3000, 10 ** 6):
        c.run(max_len=max_len)


def test_attention_scores_of_any_size():
    """Scores far from zero on both sides, equal scores, and one that outweighs all before it."""
    c = Case("f16", 2, 1, 64, 16, [1, 30], [400, 200], seed=9)
    c.q[:] = 0
    c.run()                                                     # a plain mean
    c.q[:] = 60.0
    c.k[:] = np.sign(c.k) * 50.0
    c.k[:, :, :, :, 1:] = 0
    c.run()
    c.k[:] = np.abs(c.k) * -1
    c.run()
    c = Case("f16", 2, 1, 64, 16, [1, 30], [400, 200], seed=10, sharp=0.1)
    for s in range(2):
        c.k[0][c.place(s, 150)] = 100.0
    c.q = np.abs(c.q)
    c.run()


def test_attention_infinite_values_are_seen():
    c = Case("f16", 2, 1, 64, 16, [1, 64], [100, 130], seed=11)
    c.v[0][c.place(0, 50)], c.v[0][c.place(1, 90)] = np.inf, -np.inf
    with np.errstate(all="ignore"):
        c.run()


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 bytes (k and v each): the pages lie at its end."""
    page, hk, d = 128, 8, 128
    c = Case("f16", 16, hk, d, page, [1, 5], [300, 140], seed=12)
    pages = (2 ** 32 + 2 ** 31) // (page * hk * d * 2)
    k = torch.empty((1, pages, hk, page, d), dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    at = pages - c.pages
    k[0, at:], v[0, at:] = dev(c.k[0], torch.float16), dev(c.v[0], torch.float16)
    table = np.where(c.table >= 0, c.table + at, -1)
    cache = pb.make_kv_cache(k, v)
    batch = pb.make_seq_batch(dev(c.q_start), dev(c.lens), dev(table), c.T, 5, 300)
    out = torch.empty((c.T, c.hq, d), dtype=torch.float16, device=DEV)
    lse = torch.empty((c.T, c.hq), dtype=torch.float32, device=DEV)
    ws = torch.empty(pb.pi_attention_workspace_bytes(cache, batch, c.hq), dtype=torch.uint8, device=DEV)
    q = dev(c.q, torch.float16)
    pb.pi_paged_attention(cache, 0, batch, pb.make_score_rule(c.scale), q, out, lse, ws)
    torch.cuda.synchronize()
    c.check(out.double().cpu().numpy(), lse.double().cpu().numpy())
    # the append writes there too
    new = dev(c.q[:, :hk], torch.float16)
    pb.pi_rope_append(cache, 0, batch, pb.make_rope(torch.empty(0, dtype=torch.float64, device=DEV)), None, None, new, new)
    torch.cuda.synchronize()
    for t, s, pos in R.positions(c.q_start, c.lens):
        got = v[0, int(table[s, pos // page]), :, pos % page].cpu().numpy()
        assert np.array_equal(got, c.q[t, :hk])


def test_attention_layers_streams_and_in_place():
    c = Case("f16", 4, 2, 64, 16, [2, 20], [40, 130], seed=13, layers=3, layer=2)
    c.run(stride=1)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        c.run()
    # out may be q
    k, v, q = dev(c.k, torch.float16), dev(c.v, torch.float16), dev(c.q, torch.float16)
    cache = pb.make_kv_cache(k, v)
    batch = pb.make_seq_batch(dev(c.q_start), dev(c.lens), dev(c.table), c.T, 20, 130)
    ws = torch.empty(pb.pi_attention_workspace_bytes(cache, batch, 4), dtype=torch.uint8, device=DEV)
    lse = torch.empty((c.T, 4), dtype=torch.float32, device=DEV)
    pb.pi_paged_attention(cache, 2, batch, pb.make_score_rule(c.scale), q, q, lse, ws)
    torch.cuda.synchronize()
    c.check(q.double().cpu().numpy(), lse.double().cpu().numpy())


def test_attention_random_shapes():
    rng = np.random.default_rng(14)
    for i in range(25):
        hk, g = int(rng.choice([1, 2, 3])), int(rng.choice([1, 2, 5, 8, 17]))
        d, page = int(rng.choice([16, 64, 72, 128, 192])), int(rng.choice([8, 16, 64]))
        n = int(rng.integers(1, 6))
        big = int(rng.choice([1, 4, 80]))
        new = [int(x) for x in rng.integers(0 if n > 1 else 1, big + 1, n)]
        if sum(new) == 0:
            new[0] = 1
        lens = [a + int(b) for a, b in zip(new, rng.integers(0, 400, n))]
        c = Case(str(rng.choice(["f16", "f32"])), hk * g, hk, d, page, new, lens, seed=100 + i)
        c.run(cap=float(rng.choice([0.0, 15.0])), window=int(rng.choice([0, 50])),
              slopes=slopes(hk * g) if rng.random() < 0.3 else None)


# ---- rotary positions and append -----------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d,rotary", [(64, 64), (128, 64), (80, 20), (80, 74), (96, 0), (256, 256), (8, 2)])
def test_rope_append(dtype, pairs, d, rotary):
    new, lens = [1, 5, 0, 33], [100000, 5, 3, 70]
    page, hq, hk = 16, 3, 2
    rng = np.random.default_rng(d + rotary)
    n16 = np.float16 if dtype == "f16" else np.float32
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(starts[-1])
    stride = -(-100000 // page)
    table = np.full((4, stride), -1, dtype=np.int32)
    table[0, -1] = 4                                            # only the last page of the long one is there
    table[1, 0], table[3, :5] = 9, [7, 3, 1, 0, 8]
    table[3, 3] = -1                                            # 48..63: written nowhere
    x = rng.standard_normal((T, hq + 2 * hk, d)).astype(n16)
    k0 = rng.standard_normal((2, 11, hk, page, d)).astype(n16)
    turns = pb.pi_rope_turns(rotary, 10000.0)
    m = 1.25
    for positions in (None, rng.integers(-3000, 200000, T).astype(np.int32)):
        wide = dev(x, DT[dtype])
        k, v = dev(k0, DT[dtype]), dev(k0, DT[dtype])
        cache = pb.make_kv_cache(k, v)
        batch = pb.make_seq_batch(dev(starts), dev(np.array(lens)), dev(table), T, 33, 100000)
        q, nk, nv = wide[:, :hq], wide[:, hq:hq + hk], wide[:, hq + hk:]
        q_out = torch.full((T, hq, d), 7.0, dtype=DT[dtype], device=DEV)
        rope = pb.make_rope(turns.to(DEV), pairs, m)
        pb.pi_rope_append(cache, 1, batch, rope, q, q_out, nk, nv, None if positions is None else dev(positions))
        torch.cuda.synchronize()
        rows = list(R.positions(starts, np.array(lens)))
        at = np.array([p for _, _, p in rows]) if positions is None else positions
        # sin and cos in 32 bits of an angle within 2^-24 turns; two products and a sum; one rounding
        wq, wk = R.rope(x[:, :hq], at, turns.numpy(), pairs, m), R.rope(x[:, hq:hq + hk], at, turns.numpy(), pairs, m)
        unit = 2.0 ** -11 if dtype == "f16" else 2.0 ** -24
        top = np.abs(x.astype(np.float64)).max()

        def near(got, want):
            assert (np.abs(got.astype(np.float64) - want) <= unit * np.abs(want) + 2.0 ** -20 * top + (2.0 ** -25 if dtype == "f16" else 0)).all()
        near(q_out.cpu().numpy(), wq)
        assert np.array_equal(q_out.cpu().numpy()[..., rotary:], x[:, :hq, rotary:])
        gk, gv = k.cpu().numpy(), v.cpu().numpy()
        wrote = np.zeros((11, page), dtype=bool)
        for t, s, pos in rows:
            p, i = table[s, pos // page], pos % page
            if p >= 0:
                near(gk[1, p, :, i], wk[t])
                assert np.array_equal(gk[1, p, :, i, rotary:], x[t, hq:hq + hk, rotary:])
                assert np.array_equal(gv[1, p, :, i], x[t, hq + hk:])
                wrote[p, i] = True
        for g in (gk, gv):                                      # nothing else changed
            assert np.array_equal(g[0], k0[0])
            assert np.array_equal(g[1].transpose(0, 2, 1, 3)[~wrote], k0[1].transpose(0, 2, 1, 3)[~wrote])
        # in place
        pb.pi_rope_append(cache, 1, batch, rope, q, q, nk, nv, None if positions is None else dev(positions))
        torch.cuda.synchronize()
        assert torch.equal(q, q_out)


def test_rope_keys_only_and_rows_of_nobody():
    table = np.array([[0, 1]], dtype=np.int32)
    for starts, length, want in (([0, 4], 20, [16, 17, 18, 19]), ([1, 3], 5, [3, 4]), ([0, 4], 2, [0, 1]), ([2, 2], 7, [])):
        k = torch.zeros((1, 2, 1, 16, 16), dtype=torch.float32, device=DEV)
        v = torch.zeros_like(k)
        x = torch.ones((4, 1, 16), dtype=torch.float32, device=DEV)
        batch = pb.make_seq_batch(dev(np.array(starts)), dev(np.array([length])), dev(table), 4, 4, 20)
        rope = pb.make_rope(torch.zeros(0, dtype=torch.float64, device=DEV))
        pb.pi_rope_append(pb.make_kv_cache(k, v), 0, batch, rope, None, None, x, x)
        torch.cuda.synchronize()
        hit = v[0, :, 0].reshape(32, 16).sum(1).cpu().numpy() > 0
        assert np.flatnonzero(hit).tolist() == want


# ---- pages ------------------------------------------------------------------------

def random_state(rng, pages, seqs, stride, page, share):
    """A consistent state: some sequences fork from others, some are empty."""
    refs, table, lens = np.zeros(pages, np.int32), np.full((seqs, stride), -1, np.int32), np.zeros(seqs, np.int32)
    r = R.Pages(refs, table, lens, page)
    for s in rng.permutation(seqs):
        if rng.random() < share and (r.lens > 0).any():
            r.fork([int(rng.choice(np.flatnonzero(r.lens > 0)))], [int(s)])
            r.extend([int(s)], [int(rng.integers(0, 3))])
        else:
            r.extend([int(s)], [int(rng.integers(0, stride * page // 2))])
    gone = np.flatnonzero(rng.random(seqs) < 0.3)
    r.free(gone)
    return r


def on_device(r, page):
    t = dev(r.refs), dev(r.table), dev(r.lens)
    return pb.make_page_state(*t, page), t


def same_state(t, r):
    torch.cuda.synchronize()
    for got, want, name in zip(t, (r.refs, r.table, r.lens), ("refs", "table", "lens")):
        assert np.array_equal(got.cpu().numpy(), want), name
    count = np.bincount(r.table[r.table >= 0], minlength=len(r.refs))
    assert np.array_equal(count, r.refs)                        # a state stays what it says it is


@pytest.mark.parametrize("pages,seqs,stride,page", [(1, 1, 1, 8), (40, 7, 5, 16), (500, 60, 9, 8), (9000, 300, 33, 16), (70000, 1500, 50, 32)])
def test_pages_random_steps(pages, seqs, stride, page):
    rng = np.random.default_rng(pages)
    heads, d, layers = 1, 8, 2
    with_data = pages * page < 300000
    for trial in range(3):
        r = random_state(rng, pages, seqs, stride, page, 0.5)
        st, t = on_device(r, page)
        ws = torch.full((pb.pi_pages_workspace_bytes(st, seqs),), 255, dtype=torch.uint8, device=DEV)
        k = torch.arange(layers * pages, device=DEV, dtype=torch.float32).view(layers, pages, 1, 1, 1) \
            .expand(layers, pages, heads, page, d).contiguous() if with_data else None
        v = -k if with_data else None
        cache = pb.make_kv_cache(k, v) if with_data else None
        name = np.arange(layers * pages, dtype=np.float32).reshape(layers, pages)     # what each page holds
        for step in range(3):
            n = int(rng.integers(0, seqs + 1))
            src, dst = rng.integers(-1, seqs + 1, n).astype(np.int32), rng.permutation(seqs)[:n].astype(np.int32)
            pb.pi_pages_fork(st, dev(src), dev(dst), ws)
            r.fork(src, dst)
            same_state(t, r)
            n = int(rng.integers(1, seqs + 1))
            seq = rng.permutation(seqs + 2)[:n].astype(np.int32) - 1
            seq = seq[:min(n, seqs)]
            add = rng.integers(-1, [2, 3 * page, stride * page][step] + 1, len(seq)).astype(np.int32)
            granted = torch.full((len(seq),), 9, dtype=torch.int32, device=DEV)
            copies = torch.full((2, len(seq)), 9, dtype=torch.int32, device=DEV)
            pb.pi_pages_extend(st, cache, dev(seq), dev(add), granted, copies, ws)
            want_g, want_c = r.extend(seq, add)
            same_state(t, r)
            assert np.array_equal(granted.cpu().numpy(), want_g) and np.array_equal(copies.cpu().numpy(), want_c)
            at = want_c[0] >= 0
            name[:, want_c[1][at]] = name[:, want_c[0][at]]
            gone = rng.permutation(seqs)[:int(rng.integers(0, seqs // 2 + 1))].astype(np.int32)
            pb.pi_pages_free(st, dev(gone))
            r.free(gone)
            same_state(t, r)
            if step == 1:
                moved = torch.full((pages,), 9, dtype=torch.int32, device=DEV)
                before = r.refs.copy()
                pb.pi_pages_compact(st, cache, moved, ws)
                want_m = r.compact()
                same_state(t, r)
                assert np.array_equal(moved.cpu().numpy(), want_m)
                old = name.copy()
                for p in np.flatnonzero(before > 0):
                    name[:, want_m[p]] = old[:, p]
                assert (r.refs[:int((before > 0).sum())] > 0).all()
            if with_data:
                live = r.refs > 0
                got = k.view(layers, pages, -1).cpu().numpy()
                assert (got[:, live] == name[:, live, None]).all()
                assert torch.equal(v, -k)


def test_pages_extend_runs_out_in_order():
    page = 8
    r = R.Pages(np.zeros(10, np.int32), np.full((4, 8), -1, np.int32), np.zeros(4, np.int32), page)
    st, t = on_device(r, page)
    ws = torch.empty(pb.pi_pages_workspace_bytes(st, 4), dtype=torch.uint8, device=DEV)
    g, c = torch.empty(4, dtype=torch.int32, device=DEV), torch.empty((2, 4), dtype=torch.int32, device=DEV)
    seq, add = np.array([2, 0, 3, 1], np.int32), np.array([30, 65, 50, 1], np.int32)
    # 4 pages; 9 do not fit the table; 7 are more than the 6 left; the next would fit, but its turn is after
    pb.pi_pages_extend(st, None, dev(seq), dev(add), g, c, ws)
    want, _ = r.extend(seq, add)
    same_state(t, r)
    assert g.tolist() == want.tolist() == [1, 0, 0, 0]
    add = np.array([0, 2 ** 31 - 1, 48, 0], np.int32)
    pb.pi_pages_extend(st, None, dev(seq), dev(add), g, c, ws)
    want, _ = r.extend(seq, add)
    same_state(t, r)
    assert g.tolist() == want.tolist() == [1, 0, 1, 1]


def test_pages_untrusted_ids():
    """Ids outside the pool or the table change nothing and reach no memory."""
    page = 8
    table = np.array([[5, 99, -3], [2 ** 31 - 1, -1, -1]], np.int32)
    refs, lens = np.zeros(10, np.int32), np.array([17, 3], np.int32)
    refs[5] = 1
    st, t = on_device(R.Pages(refs, table, lens, page), page)
    ws = torch.empty(pb.pi_pages_workspace_bytes(st, 2), dtype=torch.uint8, device=DEV)
    g, c = torch.empty(2, dtype=torch.int32, device=DEV), torch.empty((2, 2), dtype=torch.int32, device=DEV)
    pb.pi_pages_extend(st, None, dev(np.array([1, 2 ** 30])), dev(np.array([6, 1])), g, c, ws)
    torch.cuda.synchronize()
    assert g.tolist() == [1, 0] and c.tolist() == [[-1, -1], [-1, -1]] and t[2].tolist() == [17, 9]
    pb.pi_pages_fork(st, dev(np.array([0, 7])), dev(np.array([1, 0])), ws)
    torch.cuda.synchronize()
    assert t[1].tolist()[1] == [5, 99, -3] and t[0].tolist()[5] == 2
    pb.pi_pages_free(st, dev(np.array([1, -1])))
    torch.cuda.synchronize()
    assert t[0].tolist()[5] == 1 and t[1].tolist() == [[5, 99, -3], [-1, -1, -1]] and t[2].tolist() == [17, 0]
    moved = torch.empty(10, dtype=torch.int32, device=DEV)
    pb.pi_pages_compact(st, None, moved, ws)
    torch.cuda.synchronize()
    assert moved.tolist() == [-1] * 5 + [0] + [-1] * 4 and t[1].tolist()[0] == [0, 99, -3]


@pytest.mark.parametrize("dtype,heads,page,d,layers", [("f16", 1, 8, 8, 1), ("f32", 3, 16, 24, 3), ("f16", 8, 128, 128, 2)])
def test_pages_copy(dtype, heads, page, d, layers):
    rng = np.random.default_rng(1)
    k = torch.randn((layers, 12, heads, page, d), device=DEV).to(DT[dtype])
    v = torch.randn((layers, 12, heads, page, d), device=DEV).to(DT[dtype])
    want_k, want_v = k.clone(), v.clone()
    src, dst = np.array([3, 4, 0, -1, 12], np.int32), np.array([7, 8, 11, 2, 1], np.int32)
    for a, b in zip(src[:3], dst[:3]):
        want_k[:, b], want_v[:, b] = k[:, a], v[:, a]
    pb.pi_pages_copy(pb.make_kv_cache(k, v), dev(src), dev(dst))
    torch.cuda.synchronize()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_step_in_a_graph():
    """A step (fork, extend, append, attention) captured once and replayed: every replay gives the eager step's results."""
    rng = np.random.default_rng(2)
    page, d, hk, hq, n = 16, 64, 2, 8, 4
    r = R.Pages(np.zeros(64, np.int32), np.full((n, 8), -1, np.int32), np.zeros(n, np.int32), page)
    r.extend([0], [45])
    meta0 = dev(np.concatenate([r.refs, r.table.reshape(-1), r.lens]))
    meta = meta0.clone()
    refs, table, lens = meta[:64], meta[64:96].view(4, 8), meta[96:]
    st = pb.make_page_state(refs, table, lens, page)
    k0 = torch.randn((1, 64, hk, page, d), device=DEV).half()
    k, v = k0.clone(), k0.clone()
    cache = pb.make_kv_cache(k, v)
    batch = pb.make_seq_batch(dev(np.arange(n + 1)), lens, table, n, 1, 128)
    x = torch.randn((n, hq + 2 * hk, d), device=DEV).half()
    q, out = torch.empty((n, hq, d), dtype=torch.float16, device=DEV), torch.empty((n, hq, d), dtype=torch.float16, device=DEV)
    lse = torch.empty((n, hq), dtype=torch.float32, device=DEV)
    ws = torch.empty(max(pb.pi_pages_workspace_bytes(st, n), pb.pi_attention_workspace_bytes(cache, batch, hq)),
                     dtype=torch.uint8, device=DEV)
    g, c = torch.empty(n, dtype=torch.int32, device=DEV), torch.empty((2, n), dtype=torch.int32, device=DEV)
    src, dst, one = dev(np.zeros(n)), dev(np.arange(n)), dev(np.ones(n))
    rope, rule = pb.make_rope(pb.pi_rope_turns(d).to(DEV)), pb.make_score_rule(0.125)

    def step():
        meta.copy_(meta0)
        pb.pi_pages_fork(st, src, dst, ws)
        pb.pi_pages_extend(st, cache, dst, one, g, c, ws)
        pb.pi_rope_append(cache, 0, batch, rope, x[:, :hq], q, x[:, hq:hq + hk], x[:, hq + hk:])
        pb.pi_paged_attention(cache, 0, batch, rule, q, out, lse, ws)

    def all_of_it():
        torch.cuda.synchronize()
        return [t.clone() for t in (meta, k, v, q, out, lse, g, c)]
    step()
    want = all_of_it()
    assert want[6].tolist() == [1] * n and len(set(want[7][1].tolist())) == n
    st2 = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st2):
        step()
    for i in range(4):
        for t in (k, v, q, out, lse, g, c):
            t.copy_(k0 if t is k or t is v else torch.zeros_like(t))
        graph.replay()
        got = all_of_it()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        step()
        assert all(torch.equal(a, b) for a, b in zip(all_of_it(), want)), i
