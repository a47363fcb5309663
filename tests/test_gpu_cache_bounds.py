"""Batches and lists in device memory that are not what they should be: nothing outside the
tensors, the pages and the rows that they name is read or written."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1
# first rows that do not ascend: sequences that end before they begin, overlap, or lie outside the rows
STARTS = [[0, 9, 0, 0, 9], [5, 3, 1, 0, 9], [0, 4, 2, 9, 1], [9, 0, 9, 0, 9], [0, INT_MAX, 0, INT_MIN, 9],
          [INT_MIN, 2, INT_MIN, 5, INT_MAX], [INT_MAX, INT_MIN, INT_MAX, INT_MIN, INT_MAX], [2, INT_MIN, 4, 4, 4]]


@pytest.mark.parametrize("starts", STARTS)
def test_rope_append_first_rows_that_do_not_ascend(starts):
    """A row that its sequence does not hold is left alone, and no token is written past a sequence's length."""
    rows, page, hk, d, lens = 9, 16, 2, 16, [64, 40, 64, 20]
    table = np.arange(16, dtype=np.int32).reshape(4, 4)              # a sequence's next entry is another's page
    k = torch.zeros((1, 16, hk, page, d), dtype=torch.float32, device=DEV)
    v = torch.zeros_like(k)
    x = 1.0 + torch.rand((rows, hk, d), device=DEV)
    q_out = torch.full((rows, hk, d), 7.0, device=DEV)
    batch = pb.make_seq_batch(dev(starts), dev(lens), dev(table), rows, rows, 64)
    rope = pb.make_rope(torch.zeros(0, dtype=torch.float64, device=DEV))
    pb.pi_rope_append(pb.make_kv_cache(k, v), 0, batch, rope, x, q_out, x, x)
    torch.cuda.synchronize()
    # the sequence of a row is the one behind all those that end at or before it, if it holds the row
    held = {}
    for t in range(rows):
        s = sum(e <= t for e in starts[1:])
        if s < 4 and starts[s] <= t < starts[s + 1]:
            held[t] = (s, lens[s] - (starts[s + 1] - t))
    want = torch.zeros_like(v)
    for t, (s, pos) in held.items():
        if pos >= 0:
            want[0, int(table[s, pos // page]), :, pos % page] = x[t]
    assert torch.equal(v, want) and torch.equal(k, want)
    for t in range(rows):
        assert torch.equal(q_out[t], x[t]) if t in held else bool((q_out[t] == 7.0).all())


@pytest.mark.parametrize("starts", STARTS + [[3, INT_MIN, INT_MIN, INT_MIN, INT_MIN], [8, INT_MIN + 7, 8, INT_MIN + 8, 8]])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("group,max_new", [(1, 9), (1, 100), (8, 9)])
def test_attention_first_rows_that_do_not_ascend(starts, dtype, group, max_new):
    """Rows outside every sequence are left alone, those inside lie inside the tensors: with few rows and with many,
    split over the keys or not, whatever the workspace holds."""
    rows, page, hk, d, lens = 9, 16, 2, 64, [640, 400, 64, 2000]
    hq, stride = hk * group, 125
    table = np.arange(4 * stride, dtype=np.int32).reshape(4, stride)
    k = torch.randn((1, 4 * stride, hk, page, d), device=DEV).to(dtype)
    v = torch.ones_like(k)                                           # every weighted mean of the values is 1
    room = 40                                                        # rows on both sides that nobody may write
    q = torch.randn((rows + 2 * room, hq, d), device=DEV).to(dtype)
    out = torch.full((rows + 2 * room, hq, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((rows + 2 * room, hq), 7.0, device=DEV)
    cache = pb.make_kv_cache(k, v)
    batch = pb.make_seq_batch(dev(starts), dev(lens), dev(table), rows, max_new, 2000)
    ws = torch.full((pb.pi_attention_workspace_bytes(cache, batch, hq) // 4,), 2, dtype=torch.int32, device=DEV)
    pb.pi_paged_attention(cache, 0, batch, pb.make_score_rule(0.125), q[room:room + rows], out[room:room + rows],
                          lse[room:room + rows], ws)
    torch.cuda.synchronize()
    held = np.zeros(rows + 2 * room, dtype=bool)
    for a, b in zip(starts, starts[1:]):
        held[room + min(max(a, 0), rows):room + max(min(b, rows), 0)] |= b > a
    left = dev(~held, torch.bool)
    assert bool((out[left] == 7.0).all()) and bool((lse[left] == 7.0).all())
    sure = out[~left].double()
    assert bool(((sure - 1).abs() < 2.0 ** -9).logical_or(sure == 0).logical_or(sure == 7.0).all())
