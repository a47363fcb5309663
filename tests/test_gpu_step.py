"""Norm, microscaled projections, attention, sparse FFN and sampling together, as a decode step uses them
(sparse_activation_ffn_amd/mx.py, attention.py, examples/sample_decode.py)."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import step_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from sparse_activation_ffn_amd.attention import AttentionLayer, DecoderLayer, PagedCache  # noqa: E402
from sparse_activation_ffn_amd.layer import DeviceLayer  # noqa: E402
from sparse_activation_ffn_amd.mx import MxLinear, TokenHead  # noqa: E402
from workload import synth as S  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D, HQ, HK, HD = 256, 4, 2, 64


def host(t):
    return t.detach().cpu().numpy()


def values(mx):
    """What a matrix holds, in 64 bits."""
    return R.values(host(mx._keep[0]), host(mx._keep[1]), "fp8" if mx.format == pb.PI_MXFP8 else "fp4")


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device=DEV)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sample_decode", os.path.join(ROOT, "examples", "sample_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_linear(dtype, tokens):
    """x quantised as the definition says, then the product of what both sides hold."""
    randn = gen(tokens)
    lin = MxLinear((randn(520, 288) / 17).to(dtype), randn(520))
    x = randn(tokens, 300).to(dtype)[:, :288]                        # rows with room between them
    y = lin(x)
    torch.cuda.synchronize()
    xq = R.values(R.packed(R.codes(host(x), "fp8"), "fp8"), R.scales(host(x), "fp8"), "fp8")
    assert np.array_equal(values(lin.input.rows(tokens, DEV)), xq)
    want, tol = R.product(xq, values(lin.weight), host(lin.bias).astype(np.float64), cut=dtype == torch.float16)
    tol = tol + np.abs(want) * (2.0 ** -11 if dtype == torch.float16 else 2.0 ** -24) + 2.0 ** -25
    assert y.dtype == dtype and (np.abs(host(y).astype(np.float64) - want) <= 1.001 * tol).all()
    again = lin(lin.input.rows(tokens, DEV), dtype)                  # microscaled already
    assert torch.equal(again, y)


def test_head():
    """The last addition and norm, the vocabulary, and the draw: each step from what the one before gave."""
    randn = gen(1)
    x, delta, w = randn(9, D).half(), randn(9, D), (1 + 0.1 * randn(D)).half()
    head = TokenHead(w, MxLinear((randn(1003, D) / 4).half()))
    u = torch.rand(9, device=DEV)
    rule = pb.make_sample_rule(temperature=torch.full((9,), 0.8, device=DEV), top_k=torch.full((9,), 20, dtype=torch.int32, device=DEV))
    token = host(head(x, u, rule, delta))
    logits = host(head.logits(x, delta))
    s = R.sums(host(x), host(delta))
    y, a = R.norm(s, host(w), 1e-5), values(head.vocabulary.input.rows(9, DEV))
    # (an eighth: one step of 8 bits at most, half of one from the rounding and what a scale next door adds)
    assert (np.abs(a - y) <= np.abs(y) / 8 + 2.0 ** -9 * np.abs(y).max()).all()
    want, tol = R.product(a, values(head.vocabulary.weight), None)
    assert (np.abs(logits - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
    for i in range(9):
        t, _, _, gap = R.sample(logits[i], host(u)[i], np.float32(0.8), 20)
        assert gap > 2.0 ** -36 and token[i] == t


def layer(mx, norms, seed=0, dtype=torch.float16):
    randn = gen(seed)
    w = lambda a, b: (randn(a, b) / b ** 0.5).to(dtype)  # noqa: E731
    proj = MxLinear if mx else (lambda t: t)
    attention = AttentionLayer(proj(w((HQ + 2 * HK) * HD, D)), proj(w(D, HQ * HD)), HQ, HK, pb.make_rope(pb.pi_rope_turns(HD).to(DEV)))
    wl = S.WORKLOADS["opt30b-fp16"].scaled(d=D, n=1000, r=64)
    weights = tuple((1 + 0.1 * randn(D)).to(dtype) for _ in range(2)) if norms else None
    return DecoderLayer(attention, DeviceLayer.upload(S.make_layer(wl, layer=seed), DEV), norms=weights), weights


def run(layers, x, sizes, by_step):
    cache = PagedCache(len(layers), 40, HK, HD, 1, 200, dtype=x.dtype)
    ids, at, out = cache.ids([0]), 0, []
    for n in sizes:
        cache.extend(ids, cache.ids([n]))
        batch = cache.batch(ids, [n], at + n)
        h, delta = x[at:at + n], None
        for i, l in enumerate(layers):
            h, delta = l.step(h, delta, cache, i, batch) if by_step else (l(h, cache, i, batch), None)
        out.append(h if delta is None else (h + delta).to(x.dtype))
        at += n
    return torch.cat(out)


@pytest.mark.parametrize("mx", [False, True])
def test_layers_with_norms(mx):
    """Two layers step by step, and one call after the other, are the same but for when a sum is rounded; a layer is what its
    parts are."""
    both = [layer(mx, True, s) for s in (0, 1)]
    layers = [l for l, _ in both]
    x = gen(5)(50, D).half()
    a, b = run(layers, x, [40, 1, 9], True), run(layers, x, [40, 1, 9], False)
    # the same values are rounded, in the same places: step() keeps the FFN's output in float32 until the sum is
    assert torch.equal(a, b)
    # the second norm and the addition before it
    l, weights = both[0]
    cache = PagedCache(1, 40, HK, HD, 1, 200)
    ids = cache.ids([0])
    cache.extend(ids, cache.ids([50]))
    got, y = l.step(x, None, cache, 0, cache.batch(ids, [50], 50))
    first = R.norm(host(x), host(weights[0]), 1e-5)
    h = values(l.input.rows(50, DEV)) if mx else first
    assert (np.abs(h - first) <= np.abs(first) / 8 + 2.0 ** -9 * np.abs(first).max()).all()
    second = torch.from_numpy(R.norm(host(got), host(weights[1]), 1e-5)).to(DEV).half()
    want = l.feed_forward(second, torch.float32)
    # (an input of the FFN off by a rounding of f16 here and there)
    assert (y - want).abs().max() <= 2.0 ** -7 * want.abs().max() and y.dtype == torch.float32


def test_without_tokens_and_float32():
    l, _ = layer(True, True, 3)
    cache = PagedCache(1, 8, HK, HD, 1, 64)
    batch = cache.batch(cache.ids([]), [], 0)
    h, y = l.step(torch.empty((0, D), dtype=torch.float16, device=DEV), None, cache, 0, batch)
    assert h.shape == y.shape == (0, D)
    l, _ = layer(True, True, 4, torch.float32)
    x = gen(6)(20, D)
    out = run([l], x, [20], True)
    assert out.dtype == torch.float32 and bool(out.isfinite().all())
    parts = run([l], x, [7, 1, 12], True)
    # projections exact in float32; weights of the attention in float32: sums in other orders
    assert (out - parts).abs().max() <= 2.0 ** -3 * out.abs().max()


def test_example(example):
    """The same numbers give the same tokens; the first greedy one does not depend on them (later ones do: the FFN computes
    every token of a step over the neurons that any of them activates)."""
    model = example.Decoder(D, 1000, 64, HQ, HK, HD, 1003, 2)
    prompts = torch.randint(0, 1003, (3, 30), generator=torch.Generator().manual_seed(0)).to(DEV)
    u = torch.rand((6, 3), generator=torch.Generator().manual_seed(1)).to(DEV)
    rule = pb.make_sample_rule(temperature=torch.tensor([0.0, 0.7, 1.0], device=DEV),
                               top_p=torch.tensor([1.0, 0.9, 0.8], device=DEV))

    def tokens(p, numbers, r):
        cache = PagedCache(2, 40, HK, HD, p.shape[0], 64)
        return example.decode(model, cache, p, 6, numbers, r)
    a, b = tokens(prompts, u, rule), tokens(prompts, u, rule)
    assert torch.equal(a, b) and bool(((a >= 0) & (a < 1003)).all())
    other = tokens(prompts, torch.flip(u, [1]).contiguous(), rule)
    assert int(a[0, 0]) == int(other[0, 0])


def test_a_step_in_a_graph():
    """Norm, projection, quantisation, second product and draw captured once: every replay, on new inputs and with eager
    work between, gives what the calls give by themselves."""
    randn = gen(9)
    lin, w = MxLinear((randn(256, D) / 16).half()), (1 + 0.1 * randn(D)).half()
    head = TokenHead(w, MxLinear((randn(5003, 256) / 4).half()))
    norm, first = pb.make_norm(w), pb.empty_mx(6, D, pb.PI_MXFP8)
    rule = pb.make_sample_rule(temperature=torch.full((6,), 0.9, device=DEV), top_p=torch.full((6,), 0.9, device=DEV))
    x, delta, u = randn(6, D).half(), randn(6, D), torch.rand(6, device=DEV)
    added = torch.empty_like(x)

    def step():
        pb.pi_rms_norm(norm, x, delta=delta, sum_out=added, mx=first)
        return head(added, u, rule, lin(first))
    step()                                                           # (buffers and workspaces)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token = step()
    for i in range(6):
        x.copy_(randn(6, D).half()), delta.copy_(randn(6, D)), u.copy_(torch.rand(6, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = token.clone()
        assert torch.equal(got, step())
        randn(1000, 1000) @ randn(1000, 1000)
        torch.cuda.synchronize()


def test_a_graph_keeps_its_buffers():
    """A captured step gives the same after calls with many more rows, and after their memory's neighbours were written."""
    randn = gen(10)
    lin = MxLinear((randn(2048, 2048) / 45).half())
    head = TokenHead((1 + 0.1 * randn(2048)).half(), MxLinear((randn(1003, 2048) / 4).half()))
    x, u = randn(20, 2048).half(), torch.rand(20, device=DEV)

    def step():
        y = lin(x)
        return y, head(y, u, pb.make_sample_rule())
    want = [t.clone() for t in step()]                               # (20 rows: K is split, with a workspace)
    assert lin.ws.pieces and lin.input.codes.pieces and head.ws.pieces
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    named = [p.data_ptr() for s in (lin.ws, lin.input.codes, lin.input.scales, head.ws, head.vocabulary.input.codes) for p in s.pieces]
    for rows in (40, 64, 1000):
        head(lin(randn(rows, 2048).half()), torch.rand(rows, device=DEV))
    torch.cuda.synchronize()
    # what a freed piece would be given to
    fill = [torch.full((1 << size,), 255, dtype=torch.uint8, device=DEV) for size in range(8, 24) for _ in range(4)]
    assert not {t.data_ptr() for t in fill} & set(named)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
