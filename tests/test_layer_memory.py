"""How much the layers' buffers hold: no GPU."""
import pytest

pytest.importorskip("torch")

from sparse_activation_ffn_amd.mx import MxBuffer, Scratch  # noqa: E402


@pytest.mark.parametrize("need", [1, 257, 4097, 5_000_000, (1 << 24) + 1])
def test_a_buffer_of_one_size_holds_that(need):
    """Calls that need no more than the first hold what it needed, to the allocator's 256 bytes."""
    s = Scratch()
    for n in (need, 1, need // 2, need):
        s.bytes(n, "cpu")
    assert sum(p.numel() for p in s.pieces) == -(-need // 256) * 256


def test_growing_buffers_hold_less_than_four_times_the_need():
    """Whatever the steps in which it grows."""
    for steps in ([1000 * i for i in range(1, 200)], [256 * 2 ** i + 1 for i in range(12)], [300, 100_000, 100_001]):
        s = Scratch()
        for need in steps:
            assert s.bytes(need, "cpu").numel() >= need
        held = sum(p.numel() for p in s.pieces)
        assert held < 4 * (steps[-1] + 256) and held < 2 * s.pieces[-1].numel()


def test_activations_hold_their_rows():
    b = MxBuffer(7168)
    b.rows(1000, "cpu")
    assert sum(p.numel() for p in b.codes.pieces) == 1000 * 7168
    assert sum(p.numel() for p in b.scales.pieces) == 1000 * 224
