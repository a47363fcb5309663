"""Microscaled projections and the head over the vocabulary, driven through the C ABI:
weights in 4 bits, activations in 8, both with a scale for every 32 elements.

Only torch allocations and C calls happen here.
"""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import binding as pb


class Scratch:
    """Device memory that the calls of one stream use in turn: as much as the first needs.  For one
    that needs more there is a new piece, of twice the last one's bytes at least; the pieces before
    stay, since a captured graph may name them (all together are less than twice the last)."""

    def __init__(self):
        self.pieces = []

    def bytes(self, need: int, device) -> torch.Tensor:
        last = self.pieces[-1].numel() if self.pieces else 0
        if last < max(need, 1):
            size = max(-(-need // 256) * 256, 2 * last, 256)
            self.pieces.append(torch.empty(size, dtype=torch.uint8, device=device))
        return self.pieces[-1]


class MxBuffer:
    """Activations of up to as many rows as any call had, cols wide, in 8 bits: one step's after
    the other (calls that may overlap, on different streams, need one each)."""

    def __init__(self, cols: int, fmt: int = pb.PI_MXFP8):
        self.cols, self.fmt = cols, fmt
        self.codes, self.scales = Scratch(), Scratch()
        self.mx: Optional[pb.Mx] = None

    def rows(self, n: int, device) -> pb.Mx:
        if self.mx is None or self.mx.rows != n:
            parts = [p.bytes(n * width, device)[:n * width].view(n, width) for p, width in
                     ((self.codes, self.cols // 2 if self.fmt == pb.PI_MXFP4 else self.cols), (self.scales, self.cols // 32))]
            self.mx = pb.make_mx(*parts, self.fmt)
        return self.mx


class MxLinear:
    """y = x W^T + bias with W [n][d] (float16 or float32 device tensor, d a multiple of 32) kept in
    MXFP4; bias float32 [n] or None.  Its buffers are those of one stream: calls that may overlap
    need an MxLinear each."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None):
        n, d = weight.shape
        self.shape, self.bias = (n, d), bias
        self.weight = pb.empty_mx(n, d, pb.PI_MXFP4, weight.device)
        pb.pi_mx_quantize(weight, self.weight)
        self.input = MxBuffer(d)
        self.ws = Scratch()

    def __call__(self, x: Union[torch.Tensor, pb.Mx], dtype=None) -> torch.Tensor:
        """x [tokens][d]: float16 or float32 (rows may be strided; quantised to 8 bits here), or
        microscaled already.  The result has x's dtype, or `dtype` (float16 if x is microscaled)."""
        device = self.weight._keep[0].device
        if isinstance(x, pb.Mx):
            a, dtype = x, dtype or torch.float16
        else:
            a, dtype = self.input.rows(x.shape[0], device), dtype or x.dtype
            pb.pi_mx_quantize(x, a)
        n, d = self.shape
        need = pb.pi_mx_product_workspace_bytes(a.rows, n, d)
        ws = self.ws.bytes(need, device) if need else None
        out = torch.empty((a.rows, n), dtype=dtype, device=device)
        pb.pi_mx_product(a, self.weight, out, bias=self.bias, ws=ws)
        return out


class TokenHead:
    """From the residual stream to tokens: the last norm, the projection on the vocabulary
    (MxLinear [vocab][d]) with float32 logits, and a token drawn from each row of them."""

    def __init__(self, norm_weight: torch.Tensor, vocabulary: MxLinear, eps: float = 1e-5):
        self.norm, self.vocabulary = pb.make_norm(norm_weight, eps), vocabulary
        self.ws = Scratch()

    def logits(self, x: torch.Tensor, delta: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Of x + delta (delta: what the last layer has yet to add, see DecoderLayer.step)."""
        a = self.vocabulary.input.rows(x.shape[0], x.device)
        pb.pi_rms_norm(self.norm, x, delta=delta, mx=a)
        return self.vocabulary(a, torch.float32)

    def __call__(self, x: torch.Tensor, u: torch.Tensor, rule: Optional[pb.SampleRule] = None,
                 delta: Optional[torch.Tensor] = None) -> torch.Tensor:
        """int32 [tokens], by the random numbers u [tokens] (float32) and the rule."""
        logits = self.logits(x, delta)
        rows, vocab = logits.shape
        need = pb.pi_sample_workspace_bytes(rows, vocab)
        token = torch.empty(rows, dtype=torch.int32, device=x.device)
        pb.pi_sample(logits, rule or pb.make_sample_rule(), u, token, ws=self.ws.bytes(need, x.device))
        return token
