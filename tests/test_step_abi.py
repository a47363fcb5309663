"""Refusals of the norm, the microscaled formats and sampling: no GPU (only calls that fail validation, or have nothing
to do, are made)."""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402

FAKE = 0x10000      # never dereferenced


@pytest.fixture(scope="module")
def L():
    return pb.lib()


def ref(x):
    return None if x is None else C.byref(x)


def _mx(**kw):
    m = dict(format=pb.PI_MXFP8, rows=4, cols=128, codes=FAKE, scales=FAKE)
    m.update(kw)
    return pb.Mx(**m)


def _rows(data=FAKE, token_stride=128, head_stride=128):
    return pb.Rows(data, token_stride, head_stride)


def _norm(L, d=128, wdtype=pb.PI_F16, weight=FAKE, eps=1e-5, tokens=4, heads=1, dtype=pb.PI_F16, x=_rows(), ddtype=pb.PI_F16,
          delta=None, sum_out=None, y=_rows(FAKE << 4), mx=None, norm=True):
    n = pb.Norm(d, wdtype, weight, eps) if norm else None
    return L.pi_rms_norm(ref(n), tokens, heads, dtype, ref(x), ddtype, ref(delta), ref(sum_out), ref(y), ref(mx), None)


@pytest.mark.parametrize("kw,status", [
    (dict(norm=False), pb.PI_ERR_ARG), (dict(d=0), pb.PI_ERR_SHAPE), (dict(d=(1 << 20) + 1), pb.PI_ERR_SHAPE),
    (dict(eps=-1e-5), pb.PI_ERR_ARG), (dict(eps=math.nan), pb.PI_ERR_ARG), (dict(eps=math.inf), pb.PI_ERR_ARG),
    (dict(wdtype=pb.PI_Q4_0), pb.PI_ERR_DTYPE), (dict(weight=FAKE + 1), pb.PI_ERR_ALIGN), (dict(dtype=pb.PI_Q4_0), pb.PI_ERR_DTYPE),
    (dict(tokens=-1), pb.PI_ERR_SHAPE), (dict(heads=0), pb.PI_ERR_SHAPE), (dict(tokens=1 << 22, heads=3), pb.PI_ERR_SHAPE),
    (dict(x=None), pb.PI_ERR_ARG), (dict(x=_rows(None)), pb.PI_ERR_ARG), (dict(x=_rows(FAKE + 1)), pb.PI_ERR_ALIGN),
    (dict(x=_rows(token_stride=-1)), pb.PI_ERR_SHAPE), (dict(x=_rows(head_stride=1 << 40)), pb.PI_ERR_SHAPE),
    (dict(y=None), pb.PI_ERR_ARG), (dict(sum_out=_rows()), pb.PI_ERR_ARG), (dict(y=None, sum_out=_rows()), pb.PI_ERR_ARG),
    (dict(y=_rows(token_stride=127)), pb.PI_ERR_SHAPE), (dict(y=_rows(head_stride=100), heads=2), pb.PI_ERR_SHAPE),
    (dict(delta=_rows(), ddtype=5), pb.PI_ERR_DTYPE), (dict(delta=_rows(FAKE + 2), ddtype=pb.PI_F32), pb.PI_ERR_ALIGN),
    (dict(delta=_rows(), sum_out=_rows(FAKE << 4)), pb.PI_ERR_ARG),                     # sum and y alike
    (dict(mx=_mx(rows=5)), pb.PI_ERR_SHAPE), (dict(mx=_mx(cols=256)), pb.PI_ERR_SHAPE), (dict(mx=_mx(format=2)), pb.PI_ERR_DTYPE),
    (dict(d=120, mx=_mx(cols=96)), pb.PI_ERR_SHAPE), (dict(mx=_mx(codes=None)), pb.PI_ERR_ARG),
    (dict(tokens=0), pb.PI_OK), (dict(tokens=0, x=None), pb.PI_OK)])
def test_norm_refusals(L, kw, status):
    assert _norm(L, **kw) == status


MX_FAULTS = [(dict(format=-1), pb.PI_ERR_DTYPE), (dict(rows=-1), pb.PI_ERR_SHAPE), (dict(rows=(1 << 24) + 1), pb.PI_ERR_SHAPE),
             (dict(cols=0), pb.PI_ERR_SHAPE), (dict(cols=48), pb.PI_ERR_SHAPE), (dict(cols=(1 << 20) + 32), pb.PI_ERR_SHAPE),
             (dict(codes=None), pb.PI_ERR_ARG), (dict(scales=FAKE + 8), pb.PI_ERR_ALIGN), (dict(codes=FAKE + 4), pb.PI_ERR_ALIGN)]


@pytest.mark.parametrize("kw,status", MX_FAULTS)
def test_mx_descriptor(L, kw, status):
    m, good = _mx(**kw), _mx(format=pb.PI_MXFP4)
    assert L.pi_mx_quantize(FAKE, 128, pb.PI_F16, ref(m), None) == status
    assert L.pi_mx_dequantize(ref(m), FAKE, 128, pb.PI_F16, None) == status
    assert L.pi_mx_product(ref(m), ref(good), None, FAKE, 128, pb.PI_F16, FAKE << 8, 1 << 30, None) == status
    assert L.pi_mx_product(ref(good), ref(m), None, FAKE, 128, pb.PI_F16, FAKE << 8, 1 << 30, None) == status


def test_convert_refusals(L):
    m = _mx()
    assert L.pi_mx_quantize(FAKE, 128, pb.PI_F16, None, None) == pb.PI_ERR_ARG
    assert L.pi_mx_quantize(None, 128, pb.PI_F16, ref(m), None) == pb.PI_ERR_ARG
    assert L.pi_mx_quantize(FAKE, 128, pb.PI_Q4_0, ref(m), None) == pb.PI_ERR_DTYPE
    assert L.pi_mx_quantize(FAKE + 2, 128, pb.PI_F32, ref(m), None) == pb.PI_ERR_ALIGN
    assert L.pi_mx_quantize(FAKE, -1, pb.PI_F32, ref(m), None) == pb.PI_ERR_SHAPE
    assert L.pi_mx_dequantize(ref(m), FAKE, 127, pb.PI_F32, None) == pb.PI_ERR_SHAPE
    assert L.pi_mx_dequantize(ref(m), None, 128, pb.PI_F32, None) == pb.PI_ERR_ARG
    none = _mx(rows=0, codes=None, scales=None)
    assert L.pi_mx_quantize(None, 0, pb.PI_F16, ref(none), None) == pb.PI_OK
    assert L.pi_mx_dequantize(ref(none), None, 0, pb.PI_F16, None) == pb.PI_OK


def test_product_refusals(L):
    def call(a=_mx(), w=_mx(format=pb.PI_MXFP4, rows=256), bias=None, out=FAKE, stride=256, dtype=pb.PI_F16, ws=FAKE << 8, wsb=1 << 30):
        return L.pi_mx_product(ref(a), ref(w), bias, out, stride, dtype, ws, wsb, None)
    assert call(a=None) == pb.PI_ERR_ARG and call(w=None) == pb.PI_ERR_ARG
    assert call(w=_mx(rows=256)) == pb.PI_ERR_DTYPE                    # 8-bit weights
    assert call(a=_mx(cols=160)) == pb.PI_ERR_SHAPE
    assert call(dtype=7) == pb.PI_ERR_DTYPE
    assert call(out=None) == pb.PI_ERR_ARG
    assert call(out=FAKE + 1) == pb.PI_ERR_ALIGN
    assert call(bias=FAKE + 2) == pb.PI_ERR_ALIGN
    assert call(stride=255) == pb.PI_ERR_SHAPE
    assert call(stride=1 << 40) == pb.PI_ERR_SHAPE
    assert call(a=_mx(rows=0, codes=None, scales=None), out=None) == pb.PI_OK
    assert call(w=_mx(format=pb.PI_MXFP4, rows=0, codes=None, scales=None), out=None) == pb.PI_OK
    big = _mx(rows=4, cols=8192), _mx(format=pb.PI_MXFP4, rows=256, cols=8192)
    need = L.pi_mx_product_workspace_bytes(4, 256, 8192)
    if need:
        assert call(*big, ws=None) == pb.PI_ERR_WORKSPACE
        assert call(*big, wsb=need - 1) == pb.PI_ERR_WORKSPACE
        assert call(*big, ws=(FAKE << 8) + 16) == pb.PI_ERR_ALIGN
    for m, n, k in ((-1, 10, 64), (10, -1, 64), (10, 10, 33), (10, 10, 0), ((1 << 24) + 1, 1, 32)):
        assert L.pi_mx_product_workspace_bytes(m, n, k) == 0


def test_product_workspace_grows_with_rows(L):
    for n, k in ((1024, 8192), (7168, 8192), (50007, 1024), (64, 12288)):
        sizes = [L.pi_mx_product_workspace_bytes(m, n, k) for m in range(1, 400)] + [L.pi_mx_product_workspace_bytes(4096, n, k)]
        assert sizes == sorted(sizes)


def test_sample_refusals(L):
    need = L.pi_sample_workspace_bytes(2, 1000)
    assert need > 0

    def call(logits=FAKE, rows=2, vocab=1000, stride=1000, dtype=pb.PI_F16, rule=pb.SampleRule(), u=FAKE, token=FAKE, prob=None,
             kept=None, ws=FAKE << 8, wsb=need):
        return L.pi_sample(logits, rows, vocab, stride, dtype, ref(rule), u, token, prob, kept, ws, wsb, None)
    assert call(rule=None) == pb.PI_ERR_ARG
    for kw in (dict(rows=-1), dict(rows=65536), dict(vocab=0), dict(vocab=(1 << 20) + 1), dict(stride=-1), dict(stride=1 << 40)):
        assert call(**kw) == pb.PI_ERR_SHAPE, kw
    assert call(dtype=pb.PI_Q4_0) == pb.PI_ERR_DTYPE
    for kw in (dict(logits=None), dict(u=None), dict(token=None)):
        assert call(**kw) == pb.PI_ERR_ARG, kw
    for kw in (dict(logits=FAKE + 1), dict(u=FAKE + 1), dict(token=FAKE + 2), dict(prob=FAKE + 2), dict(kept=FAKE + 3),
               dict(rule=pb.SampleRule(temperature=FAKE + 1)), dict(rule=pb.SampleRule(top_k=FAKE + 1)),
               dict(rule=pb.SampleRule(top_p=FAKE + 1)), dict(rule=pb.SampleRule(min_p=FAKE + 1)), dict(ws=(FAKE << 8) + 16)):
        assert call(**kw) == pb.PI_ERR_ALIGN, kw
    assert call(ws=None) == pb.PI_ERR_WORKSPACE and call(wsb=need - 1) == pb.PI_ERR_WORKSPACE
    assert call(rows=0, logits=None, u=None, token=None, ws=None, wsb=0) == pb.PI_OK
    for rows, vocab in ((-1, 10), (65536, 10), (1, 0), (1, (1 << 20) + 1)):
        assert L.pi_sample_workspace_bytes(rows, vocab) == 0


def test_binding_refuses_wrong_shapes():
    """Before anything reaches the library: host tensors stand for device ones here."""
    w, x = torch.ones(64), torch.zeros((4, 64))
    n = pb.make_norm(w)
    for kw in (dict(x=torch.zeros((4, 65))), dict(y=torch.zeros((5, 64))), dict(delta=torch.zeros((4, 1, 64))),
               dict(x=torch.zeros((64, 4)).t()), dict(x=torch.zeros(64))):
        with pytest.raises(ValueError):
            pb.pi_rms_norm(n, **(dict(x=x, y=torch.zeros((4, 64))) | kw))
    with pytest.raises(TypeError):
        pb.pi_rms_norm(n, x, y=torch.zeros((4, 64), dtype=torch.float16))
    with pytest.raises(ValueError):
        pb.make_norm(torch.ones((2, 64)))
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for codes, scales, fmt in ((u8(4, 64), u8(4, 1), pb.PI_MXFP8), (u8(4, 64), u8(3, 2), pb.PI_MXFP8), (u8(4, 64), u8(4, 2), pb.PI_MXFP4),
                               (torch.zeros((4, 64)), u8(4, 2), pb.PI_MXFP8), (u8(4, 128)[:, :64], u8(4, 2), pb.PI_MXFP8)):
        with pytest.raises(ValueError):
            pb.make_mx(codes, scales, fmt)
    mx = pb.empty_mx(4, 64, pb.PI_MXFP8, "cpu")
    for bad in (torch.zeros((4, 32)), torch.zeros((64, 4)).t(), torch.zeros((4, 2, 32))):
        with pytest.raises(ValueError):
            pb.pi_mx_quantize(bad, mx)
        with pytest.raises(ValueError):
            pb.pi_mx_dequantize(mx, bad)
    wm = pb.empty_mx(10, 64, pb.PI_MXFP4, "cpu")
    with pytest.raises(ValueError):
        pb.pi_mx_product(mx, wm, torch.zeros((4, 11)))
    with pytest.raises(ValueError):
        pb.pi_mx_product(mx, wm, torch.zeros((4, 10)), bias=torch.zeros(9))
    with pytest.raises(ValueError):
        pb.make_sample_rule(top_k=torch.zeros(3))


def test_buffers_that_graphs_may_name_stay():
    """Growing buffers hand out a part of one piece, keep the pieces before it, and use less than twice the last."""
    from sparse_activation_ffn_amd.mx import MxBuffer, Scratch
    s, seen = Scratch(), []
    for need in (1, 300, 256, 5000, 4097, 70000, 3):
        t = s.bytes(need, "cpu")
        assert t.numel() >= need
        seen.append(t)
    assert {t.data_ptr() for t in seen} == {t.data_ptr() for t in s.pieces} and seen[-1] is s.pieces[-1]
    assert sum(t.numel() for t in s.pieces) < 2 * s.pieces[-1].numel()
    for fmt, width in ((pb.PI_MXFP8, 96), (pb.PI_MXFP4, 48)):
        b = MxBuffer(96, fmt)
        for n in (0, 3, 1, 200, 3):
            m = b.rows(n, "cpu")
            assert (m.rows, m.cols, m.format) == (n, 96, fmt) and m is b.rows(n, "cpu")
            assert tuple(m._keep[0].shape) == (n, width) and tuple(m._keep[1].shape) == (n, 3)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=1 << 21, heads=2, d=2056), pb.PI_ERR_SHAPE), (dict(tokens=(1 << 21) + 1, d=8192), pb.PI_ERR_SHAPE),
    # an input's place with other rows or another type
    (dict(x=_rows(token_stride=256), y=_rows()), pb.PI_ERR_ARG), (dict(x=_rows(head_stride=256), y=_rows(), heads=2), pb.PI_ERR_ARG),
    (dict(delta=_rows(FAKE << 4), ddtype=pb.PI_F32), pb.PI_ERR_ARG),
    (dict(delta=_rows(FAKE << 8), sum_out=_rows(FAKE << 8, 256)), pb.PI_ERR_ARG),
    # a microscaled output of 4 x 128 codes and 4 x 4 scales
    (dict(mx=_mx(scales=FAKE << 8)), pb.PI_ERR_ARG), (dict(mx=_mx(codes=FAKE << 8, scales=FAKE + 1008)), pb.PI_ERR_ARG),
    (dict(mx=_mx(codes=(FAKE << 4) - 496, scales=FAKE << 8)), pb.PI_ERR_ARG),
    (dict(mx=_mx(codes=FAKE << 6, scales=FAKE << 8), delta=_rows((FAKE << 8) - 1008)), pb.PI_ERR_ARG)])
def test_norm_refuses_rows_and_overlaps(L, kw, status):
    assert _norm(L, **kw) == status


def test_refusals_of_overlaps(L):
    far = FAKE << 8
    m = _mx(codes=far, scales=far << 2)                               # 4 x 128: x takes 1024 bytes of f16
    for x in (far, far + 510, far - 1022, far << 2, (far << 2) + 14, (far << 2) - 1022):
        assert L.pi_mx_quantize(x, 128, pb.PI_F16, ref(m), None) == pb.PI_ERR_ARG
        assert L.pi_mx_dequantize(ref(m), x, 128, pb.PI_F16, None) == pb.PI_ERR_ARG
    w = _mx(format=pb.PI_MXFP4, rows=256, codes=far << 4, scales=far << 6)
    for out in (far, far << 2, far << 4, far << 6, far << 8, (far << 8) + 1020):
        assert L.pi_mx_product(ref(m), ref(w), far << 8, out, 256, pb.PI_F16, None, 0, None) == pb.PI_ERR_ARG
    need = L.pi_mx_product_workspace_bytes(48, 256, 8192)
    assert need
    m, w = _mx(rows=48, cols=8192), _mx(format=pb.PI_MXFP4, rows=256, cols=8192)
    assert L.pi_mx_product(ref(m), ref(w), None, far + need - 4, 256, pb.PI_F16, far, need, None) == pb.PI_ERR_ARG
    need = L.pi_sample_workspace_bytes(2, 1000)
    at = [far * i for i in range(1, 11)]                              # logits, four lists, u, token, prob, kept, workspace

    def call(token, prob, kept):
        rule = pb.SampleRule(*at[1:5])
        return L.pi_sample(at[0], 2, 1000, 1000, pb.PI_F16, ref(rule), at[5], token, prob, kept, at[9], need, None)
    for i in (0, 1, 2, 3, 4, 5, 9):
        assert call(at[i], at[7], at[8]) == call(at[6], at[i] + 4, at[8]) == call(at[6], None, at[i]) == pb.PI_ERR_ARG
    assert call(at[6], at[6] + 4, None) == call(at[6], None, at[6]) == call(at[6], at[7], at[7] - 4) == pb.PI_ERR_ARG
