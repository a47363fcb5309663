"""A float32 step of a layer with microscaled projections, every part of it against its definition in 64 bits on what the part
before it gave: 8-bit codes next to a border and the neurons that a step's tokens activate make two ways of cutting a prompt
differ by more than any sum's order, so that whole outputs say little."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import cache_ref as C  # noqa: E402
import step_ref as R  # noqa: E402
from sparse_activation_ffn_amd import binding as pb  # noqa: E402
from sparse_activation_ffn_amd.attention import PagedCache  # noqa: E402
from test_gpu_norm_mx import check_y  # noqa: E402
from test_gpu_step import D, DEV, HD, HK, HQ, gen, host, layer, values  # noqa: E402

pytestmark = pytest.mark.gpu


def check_codes(mx, y, tol):
    """mx holds y, known within tol: half a step of 8 bits off (2^-4 of the value; 2^-10 of the scale below 2^-6 of it), cut at 448."""
    scale = np.ldexp(1.0, host(mx._keep[1]).astype(np.int64) - 127).repeat(32, -1)
    want = np.clip(y, -448 * scale, 448 * scale)
    assert (np.abs(values(mx) - want) <= np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * scale) + tol).all()
    # the scale is that of a value in tol's range
    top = np.abs(R.blocks(y)).max(-1)
    near = R.blocks(np.broadcast_to(tol, y.shape)).max(-1)
    s = np.ldexp(256.0, host(mx._keep[1]).astype(np.int64) - 127)
    assert (s <= top + near).all() and (2 * s > top - near).all()


def test_a_float32_step_part_by_part():
    l, weights = layer(True, True, 4, torch.float32)
    attention, g = l.attention, HQ // HK
    cache = PagedCache(1, 8, HK, HD, 1, 64, dtype=torch.float32)
    ids, at, keys, vals = cache.ids([0]), 0, np.zeros((0, HK, HD)), np.zeros((0, HK, HD))
    x_all, turns = gen(6)(20, D), pb.pi_rope_turns(HD).numpy()
    for n in (7, 1, 12):
        x = x_all[at:at + n].contiguous()
        cache.extend(ids, cache.ids([n]))
        got, y = l.step(x, None, cache, 0, cache.batch(ids, [n], at + n))
        torch.cuda.synchronize()
        # the first norm, rounded once
        first = l.input.rows(n, DEV)
        normed = R.norm(host(x), host(weights[0]), 1e-5)
        assert np.array_equal(host(first._keep[1]), R.scales(normed, "fp8"))
        assert np.array_equal(host(first._keep[0]), R.codes(normed, "fp8"))
        # queries, keys and values: the product is the same again, so the step's is known
        qkv = host(attention.w_qkv(first, torch.float32)).astype(np.float64)
        want, tol = R.product(values(first), values(attention.w_qkv.weight), None)
        assert (np.abs(qkv - want) <= tol + 2.0 ** -24 * np.abs(want)).all()
        # attention over all keys so far, into 8 bits
        q, k, v = np.split(qkv.reshape(n, -1, HD), [HQ, HQ + HK], 1)
        pos = np.arange(at, at + n)
        q, keys, vals = C.rope(q, pos, turns, False), np.concatenate([keys, C.rope(k, pos, turns, False)]), np.concatenate([vals, v])
        out, size = np.zeros((n, HQ, HD)), 0.0
        for i in range(n):
            for h in range(HQ):
                kk, vv = keys[:at + i + 1, h // g], vals[:at + i + 1, h // g]
                s = kk @ q[i, h] * HD ** -0.5
                w = np.exp(s - s.max())
                out[i, h] = w @ vv / w.sum()
                size = max(size, (np.abs(kk) @ np.abs(q[i, h])).max() * HD ** -0.5)
        # scores in float32: rotated keys and queries rounded (three roundings of 2^-24 each), sums and weights as in
        # cache_ref.attention_tolerance, all relative to the largest value seen
        near = (2.0 ** -24 * (80 + 12) * (1 + size) + 2.0 ** -19) * np.abs(vals).max()
        second = attention.w_o.input.rows(n, DEV)
        check_codes(second, out.reshape(n, -1), near)
        # the output projection and the addition
        want, tol = R.product(values(second), values(attention.w_o.weight), None)
        s = want + host(x).astype(np.float64)
        assert (np.abs(host(got) - s) <= tol + 2.0 ** -24 * (np.abs(want) + np.abs(s)) * 1.01).all()
        # the second norm, and the feed-forward half of what it gives
        h = torch.empty_like(got)
        pb.pi_rms_norm(l.norms[1], got, y=h)
        check_y(host(h), R.norm(host(got), host(weights[1]), 1e-5), False)
        assert torch.equal(l.feed_forward(h, torch.float32), y)
        at += n
