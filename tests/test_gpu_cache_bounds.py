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
