"""Steps of a decoder as a program makes them: 32-bit models, steps without a wait, and the sparse FFN's
maintenance between steps."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from sparse_activation_ffn_amd.attention import AttentionLayer, DecoderLayer, PagedCache  # noqa: E402
from sparse_activation_ffn_amd.layer import DeviceLayer  # noqa: E402
from workload import synth as S  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D, HQ, HK, HD = 256, 4, 2, 64


def decoder_layer(dtype=torch.float16, seed=0, n_hot=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    w = lambda a, b: (torch.randn((a, b), generator=g, device=DEV) / b ** 0.5).to(dtype)  # noqa: E731
    attention = AttentionLayer(w((HQ + 2 * HK) * HD, D), w(D, HQ * HD), HQ, HK, pb.make_rope(pb.pi_rope_turns(HD).to(DEV)))
    wl = S.WORKLOADS["opt30b-fp16"].scaled(d=D, n=1000, r=64)
    return DecoderLayer(attention, DeviceLayer.upload(S.make_layer(wl, layer=seed), DEV, n_hot=n_hot))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("tokens", [1, 63, 64, 65, 128, 150, 200])
def test_feed_forward_in_pieces(dtype, tokens):
    """Each run of 64 tokens keeps its own outputs: the same bits as the runs one by one."""
    layer = decoder_layer(dtype)
    x = torch.randn((tokens, D), device=DEV).to(dtype)
    want = torch.cat([layer.feed_forward(part).clone() for part in x.split(64)])
    assert torch.equal(layer.feed_forward(x), want)


def test_a_result_is_the_callers():
    """What a call returned is not changed by the next one."""
    layer = decoder_layer(torch.float32)
    a = layer.feed_forward(torch.randn((5, D), device=DEV))
    kept = a.clone()
    layer.feed_forward(torch.randn((5, D), device=DEV))
    assert torch.equal(a, kept)


def test_a_sequence_without_pages_leaves_the_others_alone():
    """A pool that runs dry under four beams with a shared last page: two get their pages, the others write nothing
    and see nothing until there is room again, and every token that was in the cache keeps its bits."""
    layer = decoder_layer().attention
    x = torch.randn((24, D), device=DEV).half()
    y = torch.randn((4, D), device=DEV).half()
    outs = []
    for pages in (40, 4):                                            # 24 tokens: one full page and a shared half one
        cache = PagedCache(1, pages, HK, HD, 4, 64)
        first, all4, one = cache.ids([0]), cache.ids([0, 1, 2, 3]), cache.ids([1] * 4)
        cache.extend(first, cache.ids([24]))
        layer(x, cache, 0, cache.batch(first, [24], 24))
        cache.fork(cache.ids([0] * 3), cache.ids([1, 2, 3]))
        k, v = cache.k.clone(), cache.v.clone()
        granted, copies = cache.extend(all4, one)
        out = layer(y, cache, 0, cache.batch(all4, [1] * 4, 25))
        outs.append(out)
        if pages == 40:
            assert granted.tolist() == [1] * 4
            continue
        assert granted.tolist() == [1, 1, 0, 0] and cache.lens.tolist() == [25, 25, 24, 24]
        assert torch.equal(out[:2], outs[0][:2]) and bool((out[2:] == 0).all())
        # the old pages are as they were; the copies differ from theirs at the new token alone
        old, made = copies[0, :2].long(), copies[1, :2].long()
        for now, was in ((cache.k, k), (cache.v, v)):
            same = [p for p in range(4) if p not in made.tolist()]
            assert torch.equal(now[:, same], was[:, same])
            assert torch.equal(now[:, made, :, :8], was[:, old, :, :8])
            assert torch.equal(now[:, made, :, 9:], was[:, old, :, 9:])
        # refused again, then granted once a beam has gone: as in the roomy pool
        granted, _ = cache.extend(cache.ids([2]), cache.ids([40]))
        again = layer(y[2:3], cache, 0, cache.batch(cache.ids([2]), [1], 25))
        assert granted.tolist() == [0] and bool((again == 0).all())
        cache.free(cache.ids([0]))
        granted, _ = cache.extend(cache.ids([2]), cache.ids([1]))
        again = layer(y[2:3], cache, 0, cache.batch(cache.ids([2]), [1], 25))
        assert granted.tolist() == [1] and (again - outs[0][2:3]).abs().max() < 8 * 2.0 ** -11


def test_ids_outside_the_table_take_no_part():
    layer = decoder_layer().attention
    cache = PagedCache(1, 10, HK, HD, 4, 64)
    x = torch.randn((5, D), device=DEV).half()
    cache.extend(cache.ids([0, 1]), cache.ids([5, 5]))
    layer(torch.cat([x, x]), cache, 0, cache.batch(cache.ids([0, 1]), [5, 5], 5))
    k = cache.k.clone()
    ids = cache.ids([-1, 4, 2 ** 31 - 1, 1])
    granted, _ = cache.extend(ids, cache.ids([1] * 4))
    out = layer(x[:4], cache, 0, cache.batch(ids, [1] * 4, 6))
    assert granted.tolist() == [0, 0, 0, 1] and cache.lens.tolist() == [5, 6, 0, 0]
    assert bool((out[:3] == 0).all()) and bool((out[3] != 0).any())
    changed = (cache.k != k).any(-1).any(2)[0]                        # [page][place]
    assert changed.nonzero().tolist() == [[int(cache.table[1, 0]), 5]]


def test_steps_do_not_wait():
    """A step's bookkeeping and layers only enqueue: the host is through while the stream is still at work before them."""
    layer = decoder_layer()
    cache = PagedCache(1, 40, HK, HD, 4, 100)
    x = torch.randn((4, D), device=DEV).half()

    def step(length):
        everyone = cache.ids(range(4))
        cache.fork(cache.ids([0, 0, 1, 1]), everyone)
        cache.extend(everyone, cache.ids([1] * 4))
        return layer(x, cache, 0, cache.batch(everyone, [1] * 4, length))
    for n in range(1, 4):                                            # buffers, workspaces and pinned blocks are there
        step(n)
    torch.cuda.synchronize()
    a = torch.randn((8192, 8192), device=DEV)
    done = torch.cuda.Event()
    torch.cuda.set_sync_debug_mode("error")
    try:
        for _ in range(20):                                          # 100 ms and more
            a = (a @ a).clamp_(-1, 1)
        step(4)
        step(5)
        done.record()
        assert not done.query()
    finally:
        torch.cuda.set_sync_debug_mode("default")
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [5] * 4


def test_the_example_decodes_without_a_wait():
    spec = importlib.util.spec_from_file_location("beam_decode", os.path.join(ROOT, "examples", "beam_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layers = [decoder_layer(seed=i) for i in range(2)]
    prompt = torch.randn((75, D), device=DEV).half()
    outs = []
    for mode in ("default", "error"):
        cache = PagedCache(2, 60, HK, HD, 4, 100)
        torch.cuda.set_sync_debug_mode(mode)
        try:
            outs.append(example.decode(layers, cache, prompt, 4, 7, chunk=32))
        finally:
            torch.cuda.set_sync_debug_mode("default")
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_the_ffn_may_be_maintained_between_steps(dtype):
    """After a new index, a placement on the host or a new threshold the layer runs on what its FFN holds now, for
    token counts that it has met and for others: the same bits as a layer made of the FFN as it is."""
    layer = decoder_layer(dtype, n_hot=300)
    x = torch.randn((70, D), device=DEV).to(dtype)

    def same():
        fresh = DecoderLayer(layer.attention, layer.ffn)
        for n in (1, 3, 5, 70):
            assert torch.equal(layer.feed_forward(x[:n]), fresh.feed_forward(x[:n])), n
    for n in (1, 3):
        layer.feed_forward(x[:n])
    counts = torch.randint(0, 1000, (layer.ffn.n,), dtype=torch.int32, device=DEV)
    before = layer.feed_forward(x[:3])
    layer.ffn.reindex(counts, 700, 1)                                # 700 hot rows from now on
    assert layer.ffn.n_hot == 700
    same()
    assert (layer.feed_forward(x[:3]).float() - before.float()).abs().max() < 2.0 ** -9 * before.abs().max()
    layer.ffn.place_cold_on_host()
    host = layer.ffn.cold_host["W_up"]
    host.zero_()                                                     # the rows that a step reads from now on
    torch.cuda.synchronize()
    same()
    layer.ffn.threshold = 1e9                                        # no neuron is active
    assert bool((layer.feed_forward(x[:3]) == 0).all())
    same()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_steps_without_tokens(dtype):
    """No rows at all, and sequences without new tokens among others."""
    layer = decoder_layer(dtype)
    cache = PagedCache(1, 10, HK, HD, 3, 64, dtype=dtype)
    x = torch.randn((4, D), device=DEV).to(dtype)
    none = layer(x[:0], cache, 0, cache.batch(cache.ids([]), [], 0))
    assert none.shape == (0, D) and none.dtype == dtype
    ids = cache.ids([0, 1, 2])
    cache.extend(ids, cache.ids([0, 4, 0]))
    none = layer(x[:0], cache, 0, cache.batch(ids, [0, 0, 0], 4))
    assert none.shape == (0, D)
    out = layer(x, cache, 0, cache.batch(ids, [0, 4, 0], 4))
    alone = PagedCache(1, 10, HK, HD, 1, 64, dtype=dtype)
    alone.extend(alone.ids([0]), alone.ids([4]))
    assert torch.equal(out, layer(x, alone, 0, alone.batch(alone.ids([0]), [4], 4)))
