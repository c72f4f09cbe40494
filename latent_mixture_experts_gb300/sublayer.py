"""The feed-forward half of a decoder layer: residual addition, RMS norm and a
feed-forward block - dense (GatedFFN, bf16 or MXFP8) or the MoE layer
(LatentMoE).

    y, h = sub.forward(x, residual)         # x: the output of the sublayer before
    y2, h2 = next_sub.forward(y, h)         # which adds y to the stream h

A dense bf16 sublayer trains:

    y, h, saved = sub.forward_train(x, residual)
    grads = sub.backward(dy, dh, saved)     # dh: the gradient along the stream

This module only passes buffers between the library's calls."""
from __future__ import annotations

from typing import NamedTuple

import torch

from .binding import LatentMoE
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
