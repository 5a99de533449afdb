"""Residual blocks of a sparse model on the library's kernels. With convolution:

    h = act(x W_p + b_p)                     (where the widths differ)
    y = h + ffn(norm(conv3(h)))

with ``conv3`` a 3x3x3 submanifold convolution on the sites of a kernel map,
``norm`` a layer norm and ``ffn`` a gated feed-forward block whose last product
adds the skip connection in its epilogue. With attention among an item's sites:

    h = x + attention(group_norm(x))
    h = h + attention over context(norm(h))  (where there is one)
    y = h + ffn(norm(h))

Their last products add the skip connections likewise.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import KernelMap, SubMConv3dFunction, forward
from .dense import GatedFeedForward, LayerNorm, Linear
from .packed import GroupNorm, SparseAttention

__all__ = ["SparseConvBlock", "SparseAttentionBlock"]


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


class SparseAttentionBlock(torch.nn.Module):
    """``channels``, ``hidden`` and ``groups`` as in the formulas above, ``heads``,
    ``kv_heads``, ``rotary``, ``axes`` and ``causal`` as :class:`SparseAttention`;
    ``context`` is the width of another tensor's rows that the sites attend to
    (None: no such layer). fp16 or bf16 (``dtype``), trainable. Rows are those of
    the items that ``offsets`` describe; ``positions`` [N,axes] int32 their
    coordinates, a slice of the sites' for example."""

    def __init__(self, channels: int, hidden: int, heads: int, kv_heads: Optional[int] = None, groups: int = 32,
                 context: Optional[int] = None, rotary: int = 0, axes: int = 3, causal: bool = False,
                 act: str = "silu", device=None, dtype=torch.float16):
        super().__init__()
        self.norm = GroupNorm(groups, channels, device=device)
        self.attention = SparseAttention(channels, heads, kv_heads=kv_heads, rotary=rotary, axes=axes, causal=causal,
                                         device=device, dtype=dtype)
        self.norm_context = self.over_context = None
        if context is not None:
            self.norm_context = LayerNorm(channels, device=device)
            self.over_context = SparseAttention(channels, heads, kv_heads=kv_heads, context=context, device=device,
                                                dtype=dtype)
        self.norm_ffn = LayerNorm(channels, device=device)
        self.ffn = GatedFeedForward(channels, hidden, act=act, device=device, dtype=dtype)

    def forward(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                positions: Optional[torch.Tensor] = None, context: Optional[torch.Tensor] = None,
                context_offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
        if self.over_context is None and not (context is None and context_offsets is None):
            raise ValueError("the block was made without a context")
        h = self.attention(self.norm(x, offsets), offsets, positions, residual=x)
        if self.over_context is not None:
            h = self.over_context(self.norm_context(h), offsets, context=context, context_offsets=context_offsets,
                                  residual=h)
        return self.ffn(self.norm_ffn(h), residual=h)
