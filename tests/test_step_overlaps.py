"""Refusals of operands that share memory, of the norm, the microscaled formats and sampling: no GPU (only calls that fail
validation are made)."""
import pytest

pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from test_step_abi import FAKE, L, _mx, _norm, _rows, ref  # noqa: E402,F401

FAR = FAKE << 8      # no call below reaches from FAKE to here, or from here to FAKE << 9


@pytest.mark.parametrize("tokens,heads,token_stride,head_stride", [
    (2, 2, 128, 128), (4, 3, 128, 256), (4, 3, 256, 128), (3, 64, 128 * 63, 128), (64, 3, 128, 128 * 63), (100, 100, 128 * 7, 128 * 11),
    (2, 2, 200, 300), (5, 5, 1000, 1100), (1001, 2000, 128 * 999, 128 * 1000)])
def test_norm_refuses_rows_written_over_each_other(L, tokens, heads, token_stride, head_stride):  # noqa: F811
    """Each stride holds a row, but a sum of some of them ends where another row lies."""
    rows = _rows(FAR, token_stride, head_stride)
    for dtype in (pb.PI_F16, pb.PI_F32):
        assert _norm(L, tokens=tokens, heads=heads, dtype=dtype, y=rows) == pb.PI_ERR_SHAPE
        assert _norm(L, tokens=tokens, heads=heads, dtype=dtype, y=None, sum_out=rows, delta=_rows()) == pb.PI_ERR_SHAPE
