"""A prompt and its beams through decoder layers: attention over the paged cache
and the predictor-gated sparse FFN, on synthetic weights.

The prompt goes through in chunks, forks into beams that share its pages, the
beams decode and change parents, all but one are freed, and the pages left in use
are compacted.  Bookkeeping stays on the device; only the end waits for it.

    python examples/beam_decode.py [--layers 2] [--prompt 700] [--beams 4] [--steps 16]
"""
import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from sparse_activation_ffn_amd.attention import AttentionLayer, DecoderLayer, PagedCache  # noqa: E402
from sparse_activation_ffn_amd.layer import DeviceLayer  # noqa: E402
from workload import synth as S  # noqa: E402


def make_layer(d, n, r, q_heads, kv_heads, head_dim, rope, seed, device="cuda"):
    wl = S.WORKLOADS["opt30b-fp16"].scaled(d=d, n=n, r=r)
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def weights(rows, cols):
        return (torch.randn((rows, cols), generator=g, device=device) / cols ** 0.5).half()
    attention = AttentionLayer(weights((q_heads + 2 * kv_heads) * head_dim, d), weights(d, q_heads * head_dim),
                               q_heads, kv_heads, rope)
    return DecoderLayer(attention, DeviceLayer.upload(S.make_layer(wl, layer=seed), device))


def through(layers, x, cache, batch):
    for i, layer in enumerate(layers):
        x = layer(x, cache, i, batch)
    return x


def decode(layers, cache, prompt, beams, steps, chunk=256):
    """prompt [tokens][d] -> the last step's hidden states of the beams [beams][d].  The next input of a
    beam is its last output; in every third step all beams continue the first half of them."""
    one = torch.ones(beams, dtype=torch.int32, device=prompt.device)
    first, everyone = cache.ids([0]), cache.ids(range(beams))
    length = 0
    for part in prompt.split(chunk):
        n = part.shape[0]
        cache.extend(first, cache.ids([n]))
        length += n
        x = through(layers, part, cache, cache.batch(first, [n], length))
    cache.fork(cache.ids([0] * (beams - 1)), cache.ids(range(1, beams)))
    # beams differ from here on by what they are given
    x = x[-1:] + 0.01 * torch.arange(beams, device=x.device, dtype=x.dtype)[:, None]
    for step in range(steps):
        if step % 3 == 2:
            parents = torch.div(torch.arange(beams, device=x.device), 2, rounding_mode="floor").int()
            cache.fork(parents, everyone)
            x = x[parents.long()]
        cache.extend(everyone, one)
        length += 1
        x = through(layers, x, cache, cache.batch(everyone, [1] * beams, length))
    return x


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    d, head_dim, q_heads, kv_heads = 1024, 64, 16, 4
    rope = pb.make_rope(pb.pi_rope_turns(head_dim).cuda())
    layers = [make_layer(d, 4096, 128, q_heads, kv_heads, head_dim, rope, i) for i in range(a.layers)]
    longest = a.prompt + a.steps
    pages = -(-longest // 16) + a.beams * (-(-a.steps // 16) + 2)
    cache = PagedCache(a.layers, pages, kv_heads, head_dim, a.beams, longest)
    prompt = torch.randn((a.prompt, d), device="cuda").half()
    t = time.perf_counter()
    x = decode(layers, cache, prompt, a.beams, a.steps)
    cache.free(cache.ids(range(1, a.beams)))
    cache.compact()
    used = int((cache.refs > 0).sum())
    t = time.perf_counter() - t
    assert int(cache.lens[0]) == longest, "the pool ran out of pages"
    assert used == -(-longest // 16) and bool((cache.refs[:used] == 1).all()) and bool(x.isfinite().all())
    print(f"prompt of {a.prompt}, {a.beams} beams of {a.steps} steps through {a.layers} layers in {1e3 * t:.1f} ms; "
          f"{used} of {pages} pages in use, the first {used}")


if __name__ == "__main__":
    main()
