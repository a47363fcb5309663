"""What the binding of the norm, the microscaled formats and sampling refuses of workspaces and streams: no GPU."""
import pytest

torch = pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402


def calls(ws):
    a, w = pb.empty_mx(4, 64, pb.PI_MXFP8, "cpu"), pb.empty_mx(10, 64, pb.PI_MXFP4, "cpu")
    yield lambda: pb.pi_mx_product(a, w, torch.zeros((4, 10)), ws=ws)
    yield lambda: pb.pi_sample(torch.zeros((2, 10)), pb.make_sample_rule(), torch.zeros(2), torch.zeros(2, dtype=torch.int32), ws=ws)


@pytest.mark.parametrize("ws", [torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty((64, 64), dtype=torch.uint8).t(),
                                torch.empty(1 << 20, dtype=torch.uint8)[::2]])
def test_a_workspace_is_as_long_as_it_says(ws):
    """One element repeated a million times is one byte of memory, and the library would write a million."""
    for call in calls(ws):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            call()


def test_a_stream_belongs_to_the_tensors_device(monkeypatch):
    class Stream:
        cuda_stream = 64

        def __init__(self, device_index):
            self.device_index = device_index
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert pb.stream_handle(Stream(1), 1) == 64 and pb.stream_handle(64, 1) == 64
    with pytest.raises(ValueError, match="cuda:0"):
        pb.stream_handle(Stream(0), 1)
    with pytest.raises(ValueError):
        pb.stream_handle(Stream(0), 0)
    assert pb.stream_handle(Stream(0)) == 64                         # (of calls that don't know their tensors' device)
