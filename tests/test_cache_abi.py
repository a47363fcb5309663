"""Refusals and host arithmetic of the paged cache's entry points: no GPU (only
calls that fail validation, or have nothing to do, are made)."""
import ctypes as C
import math

import numpy as np
import pytest

from sparse_activation_ffn_amd import binding as pb

FAKE = 0x10000      # never dereferenced


@pytest.fixture(scope="module")
def L():
    return pb.lib()


def _cache(**kw):
    c = dict(dtype=pb.PI_F16, layers=2, pages=10, kv_heads=2, page_size=16, head_dim=64, k=FAKE, v=FAKE)
    c.update(kw)
    return pb.KvCache(**c)


def _batch(**kw):
    b = dict(n_seqs=1, n_tokens=1, max_new=1, max_len=64, q_start=FAKE, kv_len=FAKE, table=FAKE, table_stride=4)
    b.update(kw)
    return pb.SeqBatch(**b)


def _rows(data=FAKE, token_stride=256, head_stride=64):
    return pb.Rows(data, token_stride, head_stride)


def _rule(**kw):
    r = dict(scale=1.0, cap=0.0, window=0, slopes=None, prefix=None, first=None)
    r.update(kw)
    return pb.ScoreRule(**r)


def _attn(L, cache=None, layer=0, batch=None, rule=None, q_heads=4, q=None, out=None, lse=None, ws=FAKE << 8, wsb=1 << 30):
    r = lambda x: None if x is None else C.byref(x)  # noqa: E731
    return L.pi_paged_attention(r(cache or _cache()), layer, r(batch or _batch()), r(rule or _rule()), q_heads,
                                r(q or _rows()), r(out or _rows()), lse, ws, wsb, None)


CACHE_FAULTS = [(dict(dtype=pb.PI_Q4_0), pb.PI_ERR_DTYPE), (dict(layers=0), pb.PI_ERR_SHAPE),
                (dict(pages=0), pb.PI_ERR_SHAPE), (dict(pages=(1 << 24) + 1), pb.PI_ERR_SHAPE),
                (dict(kv_heads=0), pb.PI_ERR_SHAPE), (dict(page_size=24), pb.PI_ERR_SHAPE),
                (dict(page_size=4), pb.PI_ERR_SHAPE), (dict(page_size=2048), pb.PI_ERR_SHAPE),
                (dict(head_dim=0), pb.PI_ERR_SHAPE), (dict(head_dim=60), pb.PI_ERR_SHAPE),
                (dict(head_dim=264), pb.PI_ERR_SHAPE), (dict(k=None), pb.PI_ERR_ARG),
                (dict(v=FAKE + 8), pb.PI_ERR_ALIGN)]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_descriptor(L, fault, status):
    c = _cache(**fault)
    assert _attn(L, cache=c) == status
    assert L.pi_attention_workspace_bytes(C.byref(c), C.byref(_batch()), 4) == 0
    assert L.pi_pages_copy(C.byref(c), FAKE, FAKE, 1, None) == status


@pytest.mark.parametrize("fault,status", [
    (dict(n_seqs=-1), pb.PI_ERR_SHAPE), (dict(n_tokens=-1), pb.PI_ERR_SHAPE), (dict(n_tokens=(1 << 23) + 1), pb.PI_ERR_SHAPE),
    (dict(max_new=-1), pb.PI_ERR_SHAPE), (dict(max_len=-1), pb.PI_ERR_SHAPE), (dict(table_stride=0), pb.PI_ERR_SHAPE),
    (dict(q_start=None), pb.PI_ERR_ARG), (dict(kv_len=None), pb.PI_ERR_ARG), (dict(table=FAKE + 2), pb.PI_ERR_ALIGN)])
def test_batch_descriptor(L, fault, status):
    b = _batch(**fault)
    assert _attn(L, batch=b) == status
    rope = pb.Rope(0, pb.PI_ROPE_HALVES, None, 1.0)
    assert L.pi_rope_append(C.byref(_cache()), 0, C.byref(b), C.byref(rope), None, 0, None, None,
                            C.byref(_rows()), C.byref(_rows()), None) == status


def test_attention_refusals(L):
    assert L.pi_paged_attention(None, 0, None, None, 4, None, None, None, None, 0, None) == pb.PI_ERR_ARG
    assert _attn(L, layer=2) == pb.PI_ERR_SHAPE
    assert _attn(L, layer=-1) == pb.PI_ERR_SHAPE
    assert _attn(L, q_heads=3) == pb.PI_ERR_SHAPE          # not a multiple of kv_heads
    assert _attn(L, q_heads=0) == pb.PI_ERR_SHAPE
    assert _attn(L, rule=_rule(scale=math.inf)) == pb.PI_ERR_ARG
    assert _attn(L, rule=_rule(cap=-1.0)) == pb.PI_ERR_ARG
    assert _attn(L, rule=_rule(cap=math.nan)) == pb.PI_ERR_ARG
    assert _attn(L, rule=_rule(window=-1)) == pb.PI_ERR_ARG
    assert _attn(L, rule=_rule(slopes=FAKE + 1)) == pb.PI_ERR_ALIGN
    assert _attn(L, q=_rows(None)) == pb.PI_ERR_ARG
    assert _attn(L, q=_rows(FAKE + 8)) == pb.PI_ERR_ALIGN
    assert _attn(L, out=_rows(head_stride=66)) == pb.PI_ERR_ALIGN
    assert _attn(L, out=_rows(token_stride=-256)) == pb.PI_ERR_SHAPE
    assert _attn(L, ws=None) == pb.PI_ERR_WORKSPACE
    assert _attn(L, ws=(FAKE << 8) + 16) == pb.PI_ERR_ALIGN
    need = L.pi_attention_workspace_bytes(C.byref(_cache()), C.byref(_batch()), 4)
    assert need > 0 and _attn(L, wsb=need - 1) == pb.PI_ERR_WORKSPACE
    assert b"workspace" in L.pi_last_error()


def test_nothing_to_do(L):
    """No sequences or no rows: nothing is enqueued, no pointer is needed."""
    for b in (_batch(n_seqs=0, q_start=None, kv_len=None, table=None), _batch(n_tokens=0)):
        assert _attn(L, batch=b, ws=None, wsb=0) == pb.PI_OK
        rope = pb.Rope(0, pb.PI_ROPE_HALVES, None, 1.0)
        assert L.pi_rope_append(C.byref(_cache()), 0, C.byref(b), C.byref(rope), None, 0, None, None, None, None,
                                None) == pb.PI_OK
    assert L.pi_pages_copy(C.byref(_cache()), None, None, 0, None) == pb.PI_OK


def test_rope_refusals(L):
    def call(rope=None, q_heads=4, q=_rows(), q_out=_rows(), k=_rows(), v=_rows(), positions=None):
        r = lambda x: None if x is None else C.byref(x)  # noqa: E731
        return L.pi_rope_append(C.byref(_cache()), 0, C.byref(_batch()), r(rope), positions, q_heads, r(q), r(q_out),
                                r(k), r(v), None)
    good = pb.Rope(64, pb.PI_ROPE_HALVES, FAKE, 1.0)
    assert call(None) == pb.PI_ERR_ARG
    assert call(pb.Rope(63, 0, FAKE, 1.0)) == pb.PI_ERR_SHAPE
    assert call(pb.Rope(66, 0, FAKE, 1.0)) == pb.PI_ERR_SHAPE       # over head_dim
    assert call(pb.Rope(-2, 0, FAKE, 1.0)) == pb.PI_ERR_SHAPE
    assert call(pb.Rope(64, 2, FAKE, 1.0)) == pb.PI_ERR_ARG
    assert call(pb.Rope(64, 0, None, 1.0)) == pb.PI_ERR_ARG
    assert call(pb.Rope(64, 0, FAKE + 4, 1.0)) == pb.PI_ERR_ALIGN
    assert call(good, q_heads=0) == pb.PI_ERR_SHAPE
    assert call(good, q_out=None) == pb.PI_ERR_ARG
    assert call(good, k=None) == pb.PI_ERR_ARG
    assert call(good, v=_rows(FAKE + 2)) == pb.PI_ERR_ALIGN
    assert call(good, positions=FAKE + 1) == pb.PI_ERR_ALIGN


def test_pages_refusals(L):
    def state(**kw):
        s = dict(pages=10, max_seqs=3, table_stride=4, page_size=16, refs=FAKE, table=FAKE, lens=FAKE)
        s.update(kw)
        return pb.PageState(**s)

    def extend(st, cache=None, n=1, ws=FAKE << 8, wsb=1 << 20, seqs=FAKE):
        return L.pi_pages_extend(C.byref(st), None if cache is None else C.byref(cache), seqs, FAKE, n, FAKE, FAKE, ws,
                                 wsb, None)
    for kw, status in [(dict(pages=0), pb.PI_ERR_SHAPE), (dict(max_seqs=0), pb.PI_ERR_SHAPE),
                       (dict(table_stride=0), pb.PI_ERR_SHAPE), (dict(page_size=12), pb.PI_ERR_SHAPE),
                       (dict(refs=None), pb.PI_ERR_ARG), (dict(lens=FAKE + 1), pb.PI_ERR_ALIGN)]:
        st = state(**kw)
        assert extend(st) == status
        assert L.pi_pages_fork(C.byref(st), FAKE, FAKE, 1, FAKE << 8, 1 << 20, None) == status
        assert L.pi_pages_free(C.byref(st), FAKE, 1, None) == status
        assert L.pi_pages_compact(C.byref(st), None, FAKE, FAKE << 8, 1 << 20, None) == status
    st = state()
    assert extend(st, n=4) == pb.PI_ERR_SHAPE                        # over max_seqs
    assert extend(st, seqs=None) == pb.PI_ERR_ARG
    assert extend(st, cache=_cache(pages=11)) == pb.PI_ERR_SHAPE
    assert extend(st, cache=_cache(page_size=32)) == pb.PI_ERR_SHAPE
    need = L.pi_pages_workspace_bytes(C.byref(st), 3)
    assert need > 0 and extend(st, n=3, wsb=need - 1) == pb.PI_ERR_WORKSPACE
    assert extend(st, ws=None) == pb.PI_ERR_WORKSPACE
    assert L.pi_pages_workspace_bytes(C.byref(st), 4) == 0
    assert L.pi_pages_compact(C.byref(st), None, None, FAKE << 8, 1 << 20, None) == pb.PI_ERR_ARG
    assert extend(st, n=0, seqs=None) == pb.PI_OK
    assert L.pi_pages_free(C.byref(st), None, 0, None) == pb.PI_OK


def test_rope_turns():
    d, base = 64, 10000.0
    f = base ** (-2.0 * np.arange(d // 2) / d)
    tau = 2 * math.pi
    ulp = 4 * 2.0 ** -52
    np.testing.assert_allclose(pb.pi_rope_turns(d, base).numpy() * tau, f, rtol=ulp)
    np.testing.assert_allclose(pb.pi_rope_turns(d, base, pb.PI_SCALE_LINEAR, 8.0).numpy() * tau, f / 8, rtol=ulp)
    grown = pb.pi_rope_turns(d, base, pb.PI_SCALE_BASE, 8.0).numpy() * tau
    np.testing.assert_allclose(grown[0], 1.0, rtol=ulp)
    np.testing.assert_allclose(grown[-1], f[-1] / 8, rtol=1e-13)     # 31 factors of the base's rounding
    bands = pb.pi_rope_turns(d, base, pb.PI_SCALE_BANDS, 8.0, 1.0, 4.0, 2048.0).numpy() * tau
    r = 2048.0 * f / tau
    w = np.clip((r - 1.0) / 3.0, 0.0, 1.0)
    np.testing.assert_allclose(bands, w * f + (1 - w) * f / 8, rtol=1e-13)
    np.testing.assert_allclose(bands[r >= 4], f[r >= 4], rtol=ulp)
    assert pb.pi_rope_turns(0).numel() == 0
    assert pb.pi_rope_turns(2, scaling=pb.PI_SCALE_BASE, factor=4.0).numpy() * tau == pytest.approx(1.0)
    for bad in [dict(rotary_dim=3), dict(rotary_dim=258), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, scaling=4),
                dict(rotary_dim=8, scaling=pb.PI_SCALE_LINEAR, factor=0.5), dict(rotary_dim=8, base=math.nan),
                dict(rotary_dim=8, scaling=pb.PI_SCALE_BANDS, factor=2.0, low=4.0, high=1.0, context=10.0),
                dict(rotary_dim=8, scaling=pb.PI_SCALE_BANDS, factor=2.0, context=0.0)]:
        with pytest.raises(pb.PiError):
            pb.pi_rope_turns(**bad)
