"""The feed-forward half of a decoder layer: residual addition, RMS norm and a
feed-forward block - dense (GatedFFN, bf16 or MXFP8) or the MoE layer
(LatentMoE).

    y, h = sub.forward(x, residual)         # x: the output of the sublayer before
    y2, h2 = next_sub.forward(y, h)         # which adds y to the stream h

A dense bf16 sublayer trains:

    y, h, saved = sub.forward_train(x, residual)
    grads = sub.backward(dy, dh, saved)     # dh: the gradient along the stream

GatedSublayer is the form with a norm on both sides of the block, a gate and
residual scales; it takes the block's normed input and hands on the next one's:

    n, h = sub.forward(n, h)
    n, h, saved = sub.forward_train(n, h)
    grads = sub.backward(dn, dh, saved)

The gradients of either, but for those of the inputs, lie in the order of
parameters(), which AdamW takes:

    opt = AdamW(sub.parameters())
    opt.step(grads.of_parameters())

This module only passes buffers between the library's calls."""
from __future__ import annotations

from typing import NamedTuple

import torch

from .binding import LatentMoE
from .block import lmoe_gated_add_norm, lmoe_gated_add_norm_backward
from .feed_forward import GatedFFN, lmoe_add_rms_norm, lmoe_add_rms_norm_backward


class Saved(NamedTuple):
    """What the backward pass of one batch reads."""
    h: torch.Tensor        # residual stream after the addition
    n: torch.Tensor        # its norm, the block's input
    g: torch.Tensor        # the block's pre-activations
    u: torch.Tensor


class Gradients(NamedTuple):
    dx: torch.Tensor       # of x and of the residual alike, the stream's dtype
    norm_w: torch.Tensor   # fp32
    gate: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor

    def of_parameters(self) -> list:
        return [self.norm_w, self.gate, self.up, self.down]


def _block_weights(block) -> list:
    if not isinstance(block, GatedFFN) or block.mx:
        raise ValueError("only a GatedFFN's bf16 weights are trained here")
    return [block._weights[n] for n in ("gate", "up", "down")]


class FeedForwardSublayer:
    def __init__(self, norm_w: torch.Tensor, block: GatedFFN | LatentMoE, eps: float = 1e-6):
        self.norm_w, self.block, self.eps = norm_w, block, float(eps)

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """-> (y bf16, the block's output, and h = residual + x)."""
        if isinstance(self.block, GatedFFN) and self.block.mx:
            q, s, h = lmoe_add_rms_norm(x, self.norm_w, self.eps, residual=residual, out_format="mxfp8")
            return self.block.lmoe_ffn_forward_mx(q, s), h
        n, _, h = lmoe_add_rms_norm(x, self.norm_w, self.eps, residual=residual)
        return self.block.forward(n), h

    def parameters(self) -> list:
        """norm_w and the dense block's gate, up and down."""
        return [self.norm_w, *_block_weights(self.block)]

    def _trains(self):
        if not (isinstance(self.block, GatedFFN) and self.block.training):
            raise ValueError("only a sublayer whose block is a GatedFFN made with training=True trains")

    def forward_train(self, x: torch.Tensor, residual: torch.Tensor):
        """forward of a GatedFFN made with training=True, keeping what backward reads."""
        self._trains()
        n, _, h = lmoe_add_rms_norm(x, self.norm_w, self.eps, residual=residual)
        y, g, u = self.block.lmoe_ffn_forward(n, save=True)
        return y, h, Saved(h, n, g, u)

    def backward(self, dy: torch.Tensor, dh: torch.Tensor | None, saved: Saved) -> Gradients:
        """Gradients from dy (of y, bf16) and dh (of h, its dtype; None: zero)."""
        self._trains()
        dn, dg, du, dd = self.block.lmoe_ffn_backward(saved.n, saved.g, saved.u, dy)
        dx, dw = lmoe_add_rms_norm_backward(dn, saved.h, self.norm_w, self.eps, dh=dh)
        return Gradients(dx, dw, dg, du, dd)


class GatedSaved(NamedTuple):
    """What the backward pass of one batch reads."""
    n: torch.Tensor        # the block's input
    y: torch.Tensor        # its output
    h: torch.Tensor        # residual stream after the addition
    g: torch.Tensor        # the block's pre-activations
    u: torch.Tensor


class GatedGradients(NamedTuple):
    dn: torch.Tensor                 # of the block's input, bf16
    dh: torch.Tensor                 # of the residual stream, its dtype
    post_w: torch.Tensor             # fp32
    next_w: torch.Tensor             # fp32
    res_gate: torch.Tensor | None    # fp32 [d], where there is a gate
    gate: torch.Tensor
    up: torch.Tensor
    down: torch.Tensor

    def of_parameters(self) -> list:
        norms = [self.post_w, self.next_w]
        return [*norms, *([] if self.res_gate is None else [self.res_gate]), self.gate, self.up, self.down]


class GatedSublayer:
    """A feed-forward block between norms: y = block(n), then
    h' = stream_scale * h + branch_scale * res_gate * norm(y, post_w) and
    n' = norm(h', next_w), which the next block reads.  res_gate: bf16 [d], or None.
    next_format: "bf16", or "mxfp8" where the next block is one on MXFP8 operands, whose
    input n' then is a pair (codes, scales)."""

    def __init__(self, block: GatedFFN | LatentMoE, post_w: torch.Tensor, next_w: torch.Tensor, eps: float = 1e-6,
                 res_gate: torch.Tensor | None = None, stream_scale: float = 1.0, branch_scale: float = 1.0,
                 next_format: str = "bf16"):
        if res_gate is not None and res_gate.dim() != 1:
            raise ValueError("res_gate must be [d]")
        self.block, self.post_w, self.next_w, self.eps, self.res_gate = block, post_w, next_w, float(eps), res_gate
        self.stream_scale, self.branch_scale, self.next_format = float(stream_scale), float(branch_scale), next_format

    def _next(self, y, h, fmt):
        return lmoe_gated_add_norm(y, h, self.post_w, self.next_w, self.eps, gate=self.res_gate,
                                   stream_scale=self.stream_scale, branch_scale=self.branch_scale, out_format=fmt)

    def forward(self, n, h: torch.Tensor):
        """-> (the next block's input, the stream)."""
        y = self.block.lmoe_ffn_forward_mx(*n) if isinstance(n, (tuple, list)) else self.block.forward(n)
        o, s, h = self._next(y, h, self.next_format)
        return (o if s is None else (o, s)), h

    def parameters(self) -> list:
        """post_w, next_w, res_gate where there is one, and the dense block's gate, up and down."""
        norms = [self.post_w, self.next_w]
        return [*norms, *([] if self.res_gate is None else [self.res_gate]), *_block_weights(self.block)]

    _trains = FeedForwardSublayer._trains

    def forward_train(self, n: torch.Tensor, h: torch.Tensor):
        """forward of a GatedFFN made with training=True, keeping what backward reads."""
        self._trains()
        y, g, u = self.block.lmoe_ffn_forward(n, save=True)
        o, _, h = self._next(y, h, "bf16")
        return o, h, GatedSaved(n, y, h, g, u)

    def backward(self, do: torch.Tensor, dh: torch.Tensor | None, saved: GatedSaved) -> GatedGradients:
        """Gradients from do (of the next block's input, bf16) and dh (of the stream, its dtype; None: zero)."""
        self._trains()
        d = lmoe_gated_add_norm_backward(do, saved.y, saved.h, self.post_w, self.next_w, self.eps, gate=self.res_gate,
                                         stream_scale=self.stream_scale, branch_scale=self.branch_scale, dh=dh)
        dn, dg, du, dd = self.block.lmoe_ffn_backward(saved.n, saved.g, saved.u, d.dy)
        return GatedGradients(dn, d.dresidual, d.post_w, d.next_w, d.gate, dg, du, dd)
