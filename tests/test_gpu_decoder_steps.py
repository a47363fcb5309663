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
