"""Prompts to sampled tokens on synthetic weights: microscaled projections, root-mean-square
norms that take up the residual's additions, attention over the paged cache, the
predictor-gated sparse FFN, and a token drawn from the logits of each sequence.

The prompts go through together, every sequence then decodes with rules of its own.
Nothing waits for the device until the end.

    python examples/sample_decode.py [--layers 2] [--seqs 4] [--prompt 200] [--steps 32]
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
from sparse_activation_ffn_amd.mx import MxLinear, TokenHead  # noqa: E402
from workload import synth as S  # noqa: E402


class Decoder:
    """Embedding, layers and head of a model of width d, weights drawn from a seed."""

    def __init__(self, d, n, r, q_heads, kv_heads, head_dim, vocab, layers, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weights(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) / cols ** 0.5).half()

        def norm():
            return (1 + 0.1 * torch.randn(d, generator=g, device=device)).half()
        wl = S.WORKLOADS["opt30b-fp16"].scaled(d=d, n=n, r=r)
        rope = pb.make_rope(pb.pi_rope_turns(head_dim).to(device))
        self.embedding = torch.randn((vocab, d), generator=g, device=device).half()
        self.layers = [DecoderLayer(AttentionLayer(MxLinear(weights((q_heads + 2 * kv_heads) * head_dim, d)),
                                                   MxLinear(weights(d, q_heads * head_dim)), q_heads, kv_heads, rope),
                                    DeviceLayer.upload(S.make_layer(wl, layer=i), device), norms=(norm(), norm()))
                       for i in range(layers)]
        self.head = TokenHead(norm(), MxLinear(weights(vocab, d)))

    def stream(self, tokens, cache, batch):
        """The residual stream of int tokens after all layers, and what is yet to be added to it."""
        x, delta = self.embedding[tokens.long()], None
        for i, layer in enumerate(self.layers):
            x, delta = layer.step(x, delta, cache, i, batch)
        return x, delta


def decode(model, cache, prompts, steps, u, rule):
    """prompts [seqs][tokens], u [steps][seqs] -> sampled tokens [steps][seqs]."""
    seqs, length = prompts.shape
    everyone, one = cache.ids(range(seqs)), torch.ones(seqs, dtype=torch.int32, device=prompts.device)
    cache.extend(everyone, cache.ids([length] * seqs))
    x, delta = model.stream(prompts.reshape(-1), cache, cache.batch(everyone, [length] * seqs, length))
    last = torch.arange(length - 1, seqs * length, length, device=x.device)
    out = [model.head(x[last], u[0], rule, delta[last])]
    for step in range(1, steps):
        cache.extend(everyone, one)
        length += 1
        x, delta = model.stream(out[-1], cache, cache.batch(everyone, [1] * seqs, length))
        out.append(model.head(x, u[step], rule, delta))
    return torch.stack(out)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    model = Decoder(1024, 4096, 128, 16, 4, 64, 32000, a.layers)
    longest = a.prompt + a.steps
    cache = PagedCache(a.layers, a.seqs * -(-longest // 16), 4, 64, a.seqs, longest)
    prompts = torch.randint(0, 32000, (a.seqs, a.prompt), device="cuda")
    u = torch.rand((a.steps, a.seqs), device="cuda")
    # the first sequence takes the largest logit, the others sample ever more freely
    t = torch.linspace(0, 1, a.seqs, device="cuda")
    rule = pb.make_sample_rule(temperature=t, top_k=torch.full((a.seqs,), 50, dtype=torch.int32, device="cuda"),
                               top_p=torch.full((a.seqs,), 0.95, device="cuda"))
    began = time.perf_counter()
    tokens = decode(model, cache, prompts, a.steps, u, rule).cpu()
    began = time.perf_counter() - began
    assert bool(((tokens >= 0) & (tokens < 32000)).all())
    print(f"{a.seqs} prompts of {a.prompt} and {a.steps} tokens each through {a.layers} layers in {1e3 * began:.1f} ms")


if __name__ == "__main__":
    main()
