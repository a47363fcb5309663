"""The attention half of a decoder layer over a paged key/value cache, driven
through the C ABI: the cache with its pages' bookkeeping, one layer's attention
(rotary append, then attention of the new tokens), and a whole decoder layer with
the predictor-gated sparse FFN as its other half.

Only torch allocations, plain matrix products (projections with plain weights) and C
calls happen here.  Bookkeeping stays on the device: nothing waits for a result.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple, Union

import torch

from . import binding as pb
from .layer import DeviceLayer, StepBuffers, decode_step
from .mx import MxBuffer, MxLinear, Scratch


class PagedCache:
    """Keys and values of all layers in pages, with counts, tables and lengths of up to
    max_seqs sequences (rows of the table) of up to max_len tokens."""

    def __init__(self, layers: int, pages: int, kv_heads: int, head_dim: int, max_seqs: int,
                 max_len: int, page_size: int = 16, dtype=torch.float16, device="cuda"):
        shape = (layers, pages, kv_heads, page_size, head_dim)
        self.page_size, self.max_seqs, self.device = page_size, max_seqs, device
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, **i32)
        # one more row than sequences: the place of ids outside the table, which stays empty.  room is 1 where a
        # sequence's last extension was granted
        self._table = torch.full((max_seqs + 1, -(-max_len // page_size)), -1, **i32)
        self._lens, self._room = torch.zeros(max_seqs + 1, **i32), torch.ones(max_seqs + 1, **i32)
        self._room[max_seqs] = 0
        self.table, self.lens = self._table[:max_seqs], self._lens[:max_seqs]
        self.cache = pb.make_kv_cache(self.k, self.v)
        self.state = pb.make_page_state(self.refs, self.table, self.lens, page_size)
        self.ws = torch.empty(pb.pi_pages_workspace_bytes(self.state, max_seqs),
                              dtype=torch.uint8, device=device)
        self.moved = torch.empty(pages, **i32)

    def ids(self, seqs: Sequence[int]) -> torch.Tensor:
        # from pinned memory, so that the copy is enqueued and not waited for
        return torch.tensor(list(seqs), dtype=torch.int32, pin_memory=True).to(self.device, non_blocking=True)

    def _rows(self, seqs: torch.Tensor) -> torch.Tensor:
        return seqs.clamp(-1, self.max_seqs).long()      # (-1 is the last row too)

    def extend(self, seqs: torch.Tensor, add: torch.Tensor):
        """Room for add[i] more tokens in sequence seqs[i] (int32 device tensors); a shared last
        page is copied first.  Returns (granted [n], copies [2][n]) on the device.  A sequence that
        is not granted has no part in the batches until an extension of it is."""
        n = seqs.numel()
        granted = torch.empty(n, dtype=torch.int32, device=self.device)
        copies = torch.empty((2, n), dtype=torch.int32, device=self.device)
        pb.pi_pages_extend(self.state, self.cache, seqs, add, granted, copies, self.ws)
        self._room[self._rows(seqs)] = granted
        return granted, copies

    def fork(self, src: torch.Tensor, dst: torch.Tensor):
        """Sequence dst[i] becomes what src[i] is, all at once; pages are shared."""
        pb.pi_pages_fork(self.state, src, dst, self.ws)

    def free(self, seqs: torch.Tensor):
        pb.pi_pages_free(self.state, seqs)

    def compact(self) -> torch.Tensor:
        """The pages in use move together at the head of the pool."""
        pb.pi_pages_compact(self.state, self.cache, self.moved, self.ws)
        return self.moved

    def batch(self, seqs: torch.Tensor, new: Sequence[int], max_len: int) -> pb.SeqBatch:
        """The batch of these sequences (after extend), new[i] new tokens each: rows of the step's
        tensors in this order.  max_len bounds their lengths (the host's own count of tokens).  A
        sequence whose extension was not granted has no place for its new tokens: it goes in with
        length 0, so nothing is written for it (its last places may be shared, and hold other
        tokens) and its rows see nothing."""
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        at = self._rows(seqs)
        return pb.make_seq_batch(self.ids(starts), self._lens[at] * self._room[at], self._table[at],
                                 starts[-1], max(list(new) + [0]), max_len)


class AttentionLayer:
    """One layer's attention: w_qkv [(q_heads + 2 kv_heads) * head_dim][d], w_o [d][q_heads *
    head_dim], tensors in the cache's dtype or MxLinear; rope from pb.make_rope, rule from
    pb.make_score_rule."""

    def __init__(self, w_qkv: Union[torch.Tensor, MxLinear], w_o: Union[torch.Tensor, MxLinear], q_heads: int, kv_heads: int,
                 rope: pb.Rope, rule: Optional[pb.ScoreRule] = None):
        self.q_heads, self.kv_heads = q_heads, kv_heads
        self.head_dim = w_qkv.shape[0] // (q_heads + 2 * kv_heads)
        self.w_qkv, self.w_o, self.rope = w_qkv, w_o, rope
        self.rule = rule or pb.make_score_rule(1.0 / math.sqrt(self.head_dim))
        self.ws = Scratch()

    def heads(self, x: Union[torch.Tensor, pb.Mx], dtype=None):
        """Queries, keys and values of x [tokens][d] (microscaled: for an MxLinear w_qkv, and the
        result's dtype with it): views of one product."""
        d, hq, hk = self.head_dim, self.q_heads, self.kv_heads
        y = self.w_qkv(x, dtype) if isinstance(self.w_qkv, MxLinear) else x @ self.w_qkv.t()
        y = y.view(-1, hq + 2 * hk, d)
        return y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:]

    def __call__(self, x: Union[torch.Tensor, pb.Mx], cache: PagedCache, layer: int, batch: pb.SeqBatch):
        q, k, v = self.heads(x, cache.k.dtype)
        pb.pi_rope_append(cache.cache, layer, batch, self.rope, q, q, k, v)
        need = pb.pi_attention_workspace_bytes(cache.cache, batch, self.q_heads)
        pb.pi_paged_attention(cache.cache, layer, batch, self.rule, q, q, None, self.ws.bytes(need, q.device))
        if isinstance(self.w_o, MxLinear):
            return self.w_o(q.flatten(1))                # (a view: the heads of a row lie side by side)
        return q.reshape(q.shape[0], self.q_heads * self.head_dim) @ self.w_o.t()


class DecoderLayer:
    """Attention and the predictor-gated sparse FFN, each after a norm and added to its input:
    x += attention(norm(x)); x += ffn(norm(x)).  x [tokens][d] in the cache's dtype.
    norms: the weights [d] of two root-mean-square norms, which take up the additions (step());
    without them the norms are layer norms without weights."""

    def __init__(self, attention: AttentionLayer, ffn: DeviceLayer, eps: float = 1e-5,
                 norms: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
        self.attention, self.ffn, self.eps = attention, ffn, eps
        self.buffers = {}
        self.norms = None if norms is None else tuple(pb.make_norm(w, eps) for w in norms)
        # the first norm's output goes into 8 bits where the projection after it reads them
        mx = self.norms is not None and isinstance(attention.w_qkv, MxLinear)
        self.input = MxBuffer(attention.w_qkv.shape[1]) if mx else None

    def norm(self, x: torch.Tensor) -> torch.Tensor:
        return torch.nn.functional.layer_norm(x.float(), x.shape[-1:], eps=self.eps).to(x.dtype)

    def feed_forward(self, x: torch.Tensor, dtype=None) -> torch.Tensor:
        """The sparse FFN, in runs of at most PI_MAX_BATCH tokens (a call's union of active
        neurons grows with its tokens), in x's dtype or `dtype`."""
        dtype = dtype or x.dtype
        if x.shape[0] == 0:
            return torch.empty_like(x, dtype=dtype)
        # as the FFN is now: a new index, a placement or a threshold replaces what the descriptors name
        predictor, parts = self.ffn.descriptors()
        out = []
        for part in x.split(pb.PI_MAX_BATCH):
            n = part.shape[0]
            if n not in self.buffers or self.buffers[n].lists.n_hot != self.ffn.n_hot:
                self.buffers[n] = StepBuffers(self.ffn, n, x.device)
            y = decode_step(self.ffn, part.contiguous(), self.buffers[n], predictor, parts)
            out.append(y.to(dtype, copy=True))        # (the buffers are the next run's)
        return torch.cat(out)

    def step(self, x: torch.Tensor, delta: Optional[torch.Tensor], cache: PagedCache, layer: int, batch: pb.SeqBatch):
        """The layer (of one with `norms`) on the stream x + delta (delta None: x alone): the stream
        with the attention added, and the FFN's float32 output, which the next layer's first norm
        or TokenHead adds to it."""
        h = None if self.input is not None else torch.empty_like(x)
        mx = None if self.input is None else self.input.rows(x.shape[0], x.device)
        added = None if delta is None else torch.empty_like(x)
        pb.pi_rms_norm(self.norms[0], x, delta=delta, sum_out=added, y=h, mx=mx)
        x = x if added is None else added
        a = self.attention(mx if h is None else h, cache, layer, batch)
        added, h = torch.empty_like(x), torch.empty_like(x)
        pb.pi_rms_norm(self.norms[1], x, delta=a, sum_out=added, y=h)
        return added, self.feed_forward(h, torch.float32)

    def __call__(self, x: torch.Tensor, cache: PagedCache, layer: int, batch: pb.SeqBatch):
        if self.norms is not None:
            x, y = self.step(x, None, cache, layer, batch)
            return (x + y).to(x.dtype)
        x = x + self.attention(self.norm(x), cache, layer, batch)
        return x + self.feed_forward(self.norm(x))
