"""The binding refuses tensors of the wrong type, size or layout before the library gets their addresses (no GPU:
every call here is refused)."""
import pytest

torch = pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402

T, HQ, HK, D, PAGE, PAGES, SEQS = 6, 4, 2, 16, 8, 5, 3
i32, f32, f64 = torch.int32, torch.float32, torch.float64


def z(n, dtype=i32):
    return torch.zeros(n, dtype=dtype)


@pytest.fixture
def cache():
    return pb.make_kv_cache(z((1, PAGES, HK, PAGE, D), f32), z((1, PAGES, HK, PAGE, D), f32))


@pytest.fixture
def batch():
    return pb.make_seq_batch(z(SEQS + 1), z(SEQS), z((SEQS, 4)), T, T, 32)


@pytest.fixture
def state():
    return pb.make_page_state(z(PAGES), z((SEQS, 4)), z(SEQS), PAGE)


# not int32, too short, with gaps
BAD = [lambda n: z(n, torch.int64), lambda n: z(n, f32), lambda n: z(n - 1), lambda n: z(2 * n)[::2]]
BAD_F32 = [lambda n: z(n, torch.float16), lambda n: z(n, f64), lambda n: z(n, i32), lambda n: z(n - 1, f32),
           lambda n: z(2 * n, f32)[::2]]


def attend(cache, batch, rule=None, lse=None):
    q = z((T, HQ, D), f32)
    pb.pi_paged_attention(cache, 0, batch, rule or pb.make_score_rule(1.0), q, q, lse, z(1 << 16, torch.uint8), 0)


@pytest.mark.parametrize("bad", BAD_F32)
def test_lse_and_slopes(cache, batch, bad):
    with pytest.raises(ValueError, match="lse"):
        attend(cache, batch, lse=bad(T * HQ))
    with pytest.raises(ValueError, match="slopes"):
        attend(cache, batch, pb.make_score_rule(1.0, slopes=bad(HQ)))


@pytest.mark.parametrize("bad", BAD)
def test_prefix_first_and_positions(cache, batch, bad):
    with pytest.raises(ValueError, match="prefix"):
        attend(cache, batch, pb.make_score_rule(1.0, prefix=bad(SEQS)))
    with pytest.raises(ValueError, match="first"):
        attend(cache, batch, pb.make_score_rule(1.0, first=bad(T)))
    x = z((T, HK, D), f32)
    with pytest.raises(ValueError, match="positions"):
        pb.pi_rope_append(cache, 0, batch, pb.make_rope(z(0, f64)), None, None, x, x, bad(T), 0)


@pytest.mark.parametrize("bad", [z(8, f32), z(8, torch.int64), z(16, f64)[::2]])
def test_turns(bad):
    with pytest.raises(ValueError, match="turns"):
        pb.make_rope(bad)


@pytest.mark.parametrize("bad", BAD)
def test_lists_of_the_pages_calls(cache, state, bad):
    ws, n = z(1 << 16, torch.uint8), 2
    good = dict(seqs=z(n), add=z(n), granted=z(n), copies=z((2, n)))
    for name in good:
        args = dict(good, **{name: bad(2 * n if name == "copies" else n)})
        if name == "seqs" and args["seqs"].numel() < n:
            continue                                         # (the list says how long the others are)
        with pytest.raises(ValueError, match=name):
            pb.pi_pages_extend(state, None, ws=ws, stream=0, **args)
    for name in ("src", "dst"):
        args = dict(src=z(n), dst=z(n), **{})
        args[name] = bad(n)
        if name == "src" and args["src"].numel() < n:
            continue
        with pytest.raises(ValueError, match=name):
            pb.pi_pages_fork(state, args["src"], args["dst"], ws, 0)
        with pytest.raises(ValueError, match=name):
            pb.pi_pages_copy(cache, args["src"], args["dst"], 0)
    seqs = bad(n)
    if seqs.numel() >= n:
        with pytest.raises(ValueError, match="seqs"):
            pb.pi_pages_free(state, seqs, 0)
    with pytest.raises(ValueError, match="moved"):
        pb.pi_pages_compact(state, None, bad(PAGES), ws, 0)
