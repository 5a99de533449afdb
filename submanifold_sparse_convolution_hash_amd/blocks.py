"""A residual block of a sparse model on the library's kernels:

    h = act(x W_p + b_p)                     (where the widths differ)
    y = h + ffn(norm(conv3(h)))

with ``conv3`` a 3x3x3 submanifold convolution on the sites of a kernel map,
``norm`` a layer norm and ``ffn`` a gated feed-forward block whose last product
adds the skip connection in its epilogue.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import KernelMap, SubMConv3dFunction, forward
from .dense import GatedFeedForward, LayerNorm, Linear

__all__ = ["SparseConvBlock"]


class SparseConvBlock(torch.nn.Module):
    """``channels`` and ``hidden`` as in the formulas above; ``cin`` (default:
    channels) is the width of the input rows. fp16, trainable; the convolution
    wants its channels in multiples of 8 up to 1024."""

    def __init__(self, channels: int, hidden: int, cin: Optional[int] = None, act: str = "silu", device=None):
        super().__init__()
        cin = channels if cin is None else cin
        self.proj = Linear(cin, channels, act=act, device=device) if cin != channels else None
        scale = (27 * channels) ** -0.5
        self.conv_weight = torch.nn.Parameter(
            (torch.randn(27, channels, channels, device=device) * scale).to(torch.float16))
        self.conv_bias = torch.nn.Parameter(torch.zeros(channels, device=device))
        self.norm = LayerNorm(channels, device=device)
        self.ffn = GatedFeedForward(channels, hidden, act=act, device=device)

    def forward(self, kmap: KernelMap, x: torch.Tensor) -> torch.Tensor:
        h = x if self.proj is None else self.proj(x)
        if torch.is_grad_enabled():
            c = SubMConv3dFunction.apply(h, self.conv_weight, self.conv_bias, kmap)
        else:
            c = forward(kmap, h, self.conv_weight, self.conv_bias)
        return self.ffn(self.norm(c), residual=h)
