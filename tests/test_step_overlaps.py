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


# x: 4 tokens of 128 f16 elements from FAR on, 256 bytes a row
SHIFTED = [_rows(FAR + 2), _rows(FAR - 2), _rows(FAR + 256), _rows(FAR - 256), _rows(FAR + 1022), _rows(FAR - 1022),
           _rows(FAR + 16, 256), _rows(FAR - 600, 512)]


@pytest.mark.parametrize("at", range(len(SHIFTED)))
def test_norm_refuses_outputs_that_begin_inside_an_operand(L, at):  # noqa: F811
    """Over x, over delta and over the other output, by an element, a row or the last element."""
    rows, x = SHIFTED[at], _rows(FAR)
    away = [_rows(FAR << 1), _rows(FAR << 2)]
    for kw in (dict(x=x, y=rows), dict(x=x, y=rows, delta=away[0]), dict(x=x, y=None, sum_out=rows, delta=away[0]),
               dict(x=away[0], delta=x, y=rows), dict(x=away[0], delta=x, y=away[1], sum_out=rows),
               dict(x=away[0], delta=away[1], y=x, sum_out=rows), dict(x=away[0], delta=away[1], y=rows, sum_out=x)):
        assert _norm(L, **kw) == pb.PI_ERR_ARG, kw


@pytest.mark.parametrize("ddtype", [pb.PI_F16, pb.PI_F32])
def test_norm_refuses_outputs_between_an_operands_rows(L, ddtype):  # noqa: F811
    """Heads of 64 f16 elements (128 bytes) in rows of ten heads: x takes heads 0 to 3."""
    head = 128
    x, away = _rows(FAR, 640, 64), _rows(FAR << 2, 256, 64)
    # head 3 of the same token, head 9 and thus head 0 of the next one, half a head; two heads apart from heads one apart
    for y in (_rows(FAR + 3 * head, 640, 64), _rows(FAR + 9 * head, 640, 64), _rows(FAR - head, 640, 64), _rows(FAR + 7 * head, 640, 64),
              _rows(FAR + 4 * head - 2, 640, 64), _rows(FAR + 2 * head, 640, 128), _rows(FAR + 640 * 2 * 2 + 2, 640, 64),
              _rows(FAR + 8 * head, 640, 128), _rows(FAR + 4 * head, 768, 64)):
        assert _norm(L, d=64, heads=4, x=x, y=y, delta=away, ddtype=ddtype) == pb.PI_ERR_ARG
        if ddtype == pb.PI_F16:
            assert _norm(L, d=64, heads=4, x=away, y=y, delta=x) == pb.PI_ERR_ARG
    # a delta of float32 rows, 256 bytes each in rows of 5 x 256: y among them
    for y in (_rows(FAR + 3 * 256, 640, 64), _rows(FAR + 4 * 256, 640, 128), _rows(FAR + 254, 640, 128)):
        assert _norm(L, d=64, heads=4, x=away, y=y, delta=_rows(FAR, 320, 64), ddtype=pb.PI_F32) == pb.PI_ERR_ARG


def test_norm_refuses_rows_past_addresses(L):  # noqa: F811
    far = _rows(FAR, 1 << 39)
    for kw in (dict(x=far, y=_rows()), dict(y=far), dict(delta=far), dict(sum_out=far, y=None, delta=_rows())):
        assert _norm(L, tokens=1 << 18, **kw) == pb.PI_ERR_SHAPE


@pytest.mark.parametrize("wdtype,size", [(pb.PI_F16, 2), (pb.PI_F32, 4)])
def test_norm_refuses_outputs_over_its_weight(L, wdtype, size):  # noqa: F811
    at = FAR
    kw = dict(weight=at, wdtype=wdtype)
    for rows in (_rows(at), _rows(at - 1022), _rows(at + 128 * size - 2), _rows(at - 256 * 3 + 2), _rows(at - 2048 + 128, 1024)):
        assert _norm(L, y=rows, **kw) == pb.PI_ERR_ARG
        assert _norm(L, y=None, sum_out=rows, delta=_rows(FAR << 1), **kw) == pb.PI_ERR_ARG
    # 4 x 128 codes and 4 x 4 scales
    for m in (_mx(codes=at, scales=FAR << 1), _mx(codes=at - 496, scales=FAR << 1), _mx(codes=at + 128 * size - 16, scales=FAR << 1),
              _mx(codes=FAR << 1, scales=at), _mx(codes=FAR << 1, scales=at + 128 * size - 16)):
        assert _norm(L, y=None, mx=m, **kw) == pb.PI_ERR_ARG


@pytest.mark.parametrize("fmt,size", [(pb.PI_MXFP8, 512), (pb.PI_MXFP4, 256)])
def test_codes_and_scales_that_are_written_lie_apart(L, fmt, size):  # noqa: F811
    """4 x 128 codes and 16 scales: at the same place, at the last codes, and the other way round."""
    for scales in (FAR, FAR + 16, FAR + size - 16):
        m = _mx(format=fmt, codes=FAR, scales=scales)
        assert L.pi_mx_quantize(FAR << 1, 128, pb.PI_F16, ref(m), None) == pb.PI_ERR_ARG
        assert _norm(L, y=None, mx=m) == pb.PI_ERR_ARG
    wide = _mx(format=fmt, rows=64, codes=FAR, scales=FAR - 16)          # 256 scales
    assert L.pi_mx_quantize(FAR << 1, 128, pb.PI_F16, ref(wide), None) == pb.PI_ERR_ARG
    assert _norm(L, tokens=64, y=None, mx=wide) == pb.PI_ERR_ARG


def test_sample_refuses_a_workspace_over_what_it_reads(L):  # noqa: F811
    need = L.pi_sample_workspace_bytes(2, 1000)
    at = [FAR * i for i in range(1, 10)]                             # logits, four lists, u, token, prob, kept

    def call(ws):
        rule = pb.SampleRule(*at[1:5])
        return L.pi_sample(at[0], 2, 1000, 1000, pb.PI_F16, ref(rule), at[5], at[6], at[7], at[8], ws, need, None)
    for operand in at:
        assert call(operand) == call(operand - (need - 4) // 256 * 256) == pb.PI_ERR_ARG
    assert call(at[0] + 3840) == pb.PI_ERR_ARG                       # the last of 2 x 1000 f16 logits


def test_product_refuses_a_workspace_over_what_it_reads(L):  # noqa: F811
    at = [FAR * 64 * i for i in range(1, 7)]                         # codes and scales of a and of w, bias, out
    a, w = _mx(rows=48, cols=8192, codes=at[0], scales=at[1]), _mx(format=pb.PI_MXFP4, rows=256, cols=8192, codes=at[2], scales=at[3])
    need = L.pi_mx_product_workspace_bytes(48, 256, 8192)
    assert need and need % 256 == 0
    sizes = (48 * 8192, 48 * 256, 256 * 4096, 256 * 256, 1024)
    for operand, size in zip(at, sizes):
        for ws in (operand, operand - need + 256, operand + size - 256):
            assert L.pi_mx_product(ref(a), ref(w), at[4], at[5], 256, pb.PI_F32, ws, need, None) == pb.PI_ERR_ARG
