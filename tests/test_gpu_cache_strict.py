"""The attention tests of test_gpu_cache.py with a comparison that no NaN passes, and batches of more
than 64 sequences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_ref as R  # noqa: E402
import cache_strict  # noqa: E402
import test_gpu_cache as G  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402
# collected here again, under the comparison that the fixture below sets
from test_gpu_cache import (test_attention_bounds_are_hints, test_attention_caps, test_attention_chunks,  # noqa: E402,F401
                            test_attention_entries_that_name_no_page, test_attention_extreme_bounds,
                            test_attention_f32_tiles_of_few_rows, test_attention_infinite_values_are_seen,
                            test_attention_layers_streams_and_in_place, test_attention_long,
                            test_attention_masked_values_have_no_influence, test_attention_offsets_past_32_bits,
                            test_attention_random_shapes, test_attention_rows_that_see_nothing, test_attention_rules,
                            test_attention_scores_of_any_size, test_attention_single_tokens, test_attention_untrusted_counts)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(G.Case, "check", cache_strict.check)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n", [64, 65, 200])
@pytest.mark.parametrize("most", [1, 40])
def test_attention_many_sequences(dtype, n, most):
    """The search for a row's sequence goes on past its first 64; empty ones and long ones among them."""
    rng = np.random.default_rng(n)
    new = [1] * n if most == 1 else [int(x) for x in rng.choice([0, 1, 2, 9, most], n)]
    lens = [a + int(b) for a, b in zip(new, rng.integers(0, 120, n))]
    lens[70 % n] += 2500
    G.Case(dtype, 4, 1, 64, 16, new, lens, seed=n).run()


@pytest.mark.parametrize("n", [64, 65, 200])
def test_rope_append_many_sequences(n):
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.choice([0, 1, 2, 9], n)]
    lens = [a + int(b) for a, b in zip(new, rng.integers(0, 40, n))]
    c = G.Case("f32", 1, 1, 16, 8, new, lens, seed=n)
    k, v = G.dev(c.k, torch.float32), G.dev(c.v, torch.float32)
    batch = pb.make_seq_batch(G.dev(c.q_start), G.dev(c.lens), G.dev(c.table), c.T, 9, max(lens))
    x = c.rng.standard_normal((c.T, 1, 16)).astype(np.float32)
    rope = pb.make_rope(torch.zeros(0, dtype=torch.float64, device=G.DEV))
    pb.pi_rope_append(pb.make_kv_cache(k, v), 0, batch, rope, None, None, G.dev(x, torch.float32), G.dev(x, torch.float32))
    torch.cuda.synchronize()
    want = c.v[0].copy()
    for t, s, pos in R.positions(c.q_start, c.lens):
        want[c.place(s, pos)] = x[t]
    assert np.array_equal(v[0].cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("hq,hk,d,new,lens", [(8, 1, 128, [1, 1], [9001, 700]), (2, 2, 64, [1], [20000]), (4, 2, 80, [6], [7000]),
                                              (2, 1, 64, [100, 1], [5000, 3000]), (2, 1, 256, [70], [3000])])
def test_attention_masked_values_in_splits(dtype, hq, hk, d, new, lens):
    """Junk that no row sees, in pieces of the keys where some rows see nothing at all, stays out of the joins."""
    c = G.Case(dtype, hq, hk, d, 16, new, lens, seed=30)
    c.k[:, c.free], c.v[:, c.free] = np.nan, np.inf
    for s, n in enumerate(lens):
        used = n % 16
        if used:
            c.k[0, c.table[s, (n - 1) // 16], :, used:], c.v[0, c.table[s, (n - 1) // 16], :, used:] = np.nan, -np.inf
        for j in range(1000 if n > 2000 else 200):                    # before the first key of every row
            p = c.place(s, j)
            c.k[0][p], c.v[0][p] = np.inf, np.nan
    rows = list(R.positions(c.q_start, c.lens))
    lowest = np.array([1000 if lens[s] > 2000 else 200 for _, s, _ in rows])
    c.run(first=lowest)
    # every second row sees its last keys alone, the rows between them everything from the lowest on
    c.run(first=np.where(np.arange(c.T) % 2 == 0, np.array([p for _, _, p in rows]) - 2, lowest))
    c.run(first=lowest, window=300)
