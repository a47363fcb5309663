"""Lengths at the ends of what a sequence may hold (2^30 tokens)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 1 << 30


@pytest.mark.parametrize("length,add,ok", [
    (LIMIT - 5, 5, 1), (LIMIT - 5, 6, 0), (LIMIT, 0, 1), (LIMIT, 1, 0), (LIMIT - 1024, 1024, 1), (LIMIT - 1024, 1025, 0),
    (2 ** 31 - 9, 8, 0), (2 ** 31 - 9, 100, 0), (2 ** 31 - 1, 2 ** 31 - 1, 0), (5, 2 ** 31 - 1, 0)])
def test_extend_stops_at_the_longest_sequence(length, add, ok):
    """A table wide enough for 2^31 tokens: growth past 2^30, where append and attention end, is not granted."""
    page, stride = 1024, 1 << 21
    i32 = dict(dtype=torch.int32, device=DEV)
    refs, table = torch.zeros(40, **i32), torch.full((2, stride), -1, **i32)
    lens = torch.tensor([length, 7], **i32)
    refs[3], table[1, 0] = 1, 3
    st = pb.make_page_state(refs, table, lens, page)
    ws = torch.empty(pb.pi_pages_workspace_bytes(st, 2), dtype=torch.uint8, device=DEV)
    g, c = torch.empty(2, **i32), torch.empty((2, 2), **i32)
    pb.pi_pages_extend(st, None, torch.tensor([0, 1], **i32), torch.tensor([add, 1], **i32), g, c, ws)
    torch.cuda.synchronize()
    grown = -(-(length + add) // page) - -(-length // page) if ok else 0
    assert g.tolist() == [ok, 1] and lens.tolist() == [length + add if ok else length, 8]
    assert int((refs > 0).sum()) == 1 + grown and int((table[0] >= 0).sum()) == grown


def test_a_sequence_named_again_and_again_stays_in_its_row():
    """A list that names one sequence more than once is not what the call asks for, but no other row is written."""
    page, stride, seqs, n = 1024, 1 << 20, 2100, 2100
    i32 = dict(dtype=torch.int32, device=DEV)
    refs, lens = torch.zeros(1 << 22, **i32), torch.zeros(seqs, **i32)
    table = torch.full((seqs, stride), -1, **i32)
    st = pb.make_page_state(refs, table, lens, page)
    ws = torch.empty(pb.pi_pages_workspace_bytes(st, n), dtype=torch.uint8, device=DEV)
    ids, add = torch.full((n,), -1, **i32), torch.zeros(n, **i32)
    for i in (3, 3 + 1024, 3 + 2048):                                # in passes of their own, each grown by the one before
        ids[i], add[i] = 5, LIMIT
    g, c = torch.empty(n, **i32), torch.empty((2, n), **i32)
    pb.pi_pages_extend(st, None, ids, add, g, c, ws)
    torch.cuda.synchronize()
    assert int(g.sum()) == 3
    for s in (0, 1, 2, 3, 4, 6, 7, 8):
        assert bool((table[s] == -1).all()), s
