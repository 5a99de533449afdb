"""Operators on the rows of items packed one after the other: group norm with an
activation, rotary positions and attention among the rows of an item, forward
and backward, on the library's kernels.

A batch of items is its rows and their ``offsets``, [items + 1] int32 on the
device, ascending from 0: item b has the rows ``offsets[b]`` to ``offsets[b + 1]
- 1`` (:func:`item_offsets` finds them from sites' coordinates). ``None`` is one
item of all rows. Rows from ``offsets[-1]`` on belong to no item and come out as
zeros. Offsets stay on the device and are not checked there beyond never leaving
the tensors: they must ascend.

The functions compute without recording gradients; the ``*Function`` classes and
the modules are the autograd form.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _DTYPES, SubmconvError
from .dense import (_INT32_MAX, _NORM_DTYPES, Linear, _act, _call, _dense, _optional, _ptr, _recorded, _rows,
                    _workspace)

__all__ = [
    "item_offsets", "group_norm", "group_norm_backward", "rotary", "rotary_frequencies", "attention",
    "attention_backward", "GroupNormFunction", "RotaryFunction", "AttentionFunction", "GroupNorm", "SparseAttention",
]

_MOST_ITEMS = 65535


def item_offsets(coords: torch.Tensor, batch: Optional[int] = None) -> torch.Tensor:
    """Row offsets [batch + 1] int32 of the items of sites ``coords`` ([N,4] int32
    (b,x,y,z), device, rows in the order of their item). Waits for the stream
    (validation); an item may have no rows."""
    if not isinstance(coords, torch.Tensor):
        raise TypeError("coords must be a tensor")
    if coords.device.type != "cuda":
        raise ValueError(f"coords must be a device tensor, got {coords.device}")
    if coords.dtype != torch.int32:
        raise TypeError(f"coords must be {torch.int32}, got {coords.dtype}")
    if coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError(f"coords must be [N,4], got {tuple(coords.shape)}")
    n = coords.shape[0]
    if batch is None:
        batch = int(coords[:, 0].max().item()) + 1 if n else 1
    else:
        batch = _count(batch, "batch")
    if not 1 <= batch <= _MOST_ITEMS:  # before there is memory for them
        raise SubmconvError(-1, f"{batch} items, 1 to {_MOST_ITEMS} are supported")
    out = coords.new_empty((batch + 2,))
    _call(coords.device, "submconv_item_offsets", _ptr(coords), coords.stride(0), n, batch, _ptr(out),
          out[-1:].data_ptr())
    bad = int(out[-1].item())
    if bad & 1:
        raise SubmconvError(-1, f"coords: a batch index outside 0 .. {batch - 1}")
    if bad:
        raise SubmconvError(-1, "coords: rows are not in the order of their items")
    return out[:-1]


def _count(v, name: str) -> int:
    v = int(v)
    if not 0 <= v <= _INT32_MAX:
        raise ValueError(f"{name} is {v}")
    return v


def _items(offsets, name: str, device) -> int:
    """Checks offsets and returns the number of items."""
    if offsets is None:
        return 1
    if not isinstance(offsets, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"{name} must be [items + 1], got {tuple(offsets.shape)}")
    if offsets.dtype != torch.int32:
        raise TypeError(f"{name} must be {torch.int32}, got {offsets.dtype}")
    if offsets.device != device:
        raise ValueError(f"{name} is on {offsets.device}, not on {device}")
    if not offsets.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return offsets.shape[0] - 1


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------


def _groups(groups, c: int) -> int:
    g = _count(groups, "groups")
    if g < 1 or c % g:
        raise ValueError(f"{c} channels do not make {g} groups")
    return g


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, act: Optional[str] = None,
               offsets: Optional[torch.Tensor] = None, return_stats: bool = False):
    """``act(group_norm(x))`` per item over its rows and each group of C / groups
    neighbouring channels: ``x`` [N,C] (fp16, bf16 or fp32; C up to 8192; rows of a
    wider tensor are fine), fp32 ``weight`` and ``bias`` ([C], either may be None),
    ``act`` one of :data:`ACTIVATIONS`. ``y`` in x's dtype, or ``(y, mean, rstd)``
    with the fp32 statistics [items,groups] that :func:`group_norm_backward`
    takes (of an empty item 0 and 1 / sqrt(eps))."""
    ld = _rows(x, "x", _NORM_DTYPES)
    n, c = x.shape
    dev = x.device
    g = _groups(groups, c)
    items = _items(offsets, "offsets", dev)
    _optional(weight, "weight", torch.float32, (c,), dev)
    _optional(bias, "bias", torch.float32, (c,), dev)
    a = _act(act)
    dt = _NORM_DTYPES[x.dtype]
    y = x.new_empty((n, c))
    mean = rstd = None
    if return_stats:
        mean = x.new_empty((items, g), dtype=torch.float32)
        rstd = x.new_empty((items, g), dtype=torch.float32)
    ws, nb = _workspace("submconv_group_norm_workspace_bytes", x, n, c, g, items, dt)
    _call(dev, "submconv_group_norm", _ptr(x), ld, n, c, g, _ptr(offsets), items, _ptr(weight), _ptr(bias), eps, a,
          _ptr(y), _ptr(mean), _ptr(rstd), dt, _ptr(ws), nb)
    return (y, mean, rstd) if return_stats else y


def group_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        act: Optional[str] = None, offsets: Optional[torch.Tensor] = None, needs=(True, True, True)):
    """``(grad_x, grad_weight, grad_bias)`` of :func:`group_norm`: grad_x in x's
    dtype, the others fp32 [C]. ``mean`` and ``rstd`` as the forward returned them;
    ``bias`` is read where there is an activation. ``needs`` leaves gradients out
    (None)."""
    ldx = _rows(x, "x", _NORM_DTYPES)
    n, c = x.shape
    dev = x.device
    ldg = _rows(grad_out, "grad_out", (x.dtype,), c, x)
    items = _items(offsets, "offsets", dev)
    if not isinstance(mean, torch.Tensor) or mean.dim() != 2:
        raise ValueError("mean must be [items,groups]")
    g = _groups(mean.shape[1], c)
    _dense(mean, "mean", torch.float32, (items, g), dev)
    _dense(rstd, "rstd", torch.float32, (items, g), dev)
    _optional(weight, "weight", torch.float32, (c,), dev)
    _optional(bias, "bias", torch.float32, (c,), dev)
    a = _act(act)
    dt = _NORM_DTYPES[x.dtype]
    gx = x.new_empty((n, c)) if needs[0] else None
    gw = x.new_empty((c,), dtype=torch.float32) if needs[1] else None
    gb = x.new_empty((c,), dtype=torch.float32) if needs[2] else None
    ws, nb = _workspace("submconv_group_norm_backward_workspace_bytes", x, n, c, g, items, dt)
    _call(dev, "submconv_group_norm_backward", _ptr(grad_out), ldg, _ptr(x), ldx, n, c, g, _ptr(offsets), items,
          _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(bias), a, _ptr(gx), _ptr(gw), _ptr(gb), dt, _ptr(ws), nb)
    return gx, gw, gb


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------


def _heads(t, name: str, dtypes, like=None) -> Tuple[int, int]:
    """Checks rows of heads [N,H,D] and returns their strides (row, head)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims (rows, heads, columns), got {tuple(t.shape)}")
    n, h, d = shape = t.shape
    if like is not None:
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")
        if shape != like.shape:
            raise ValueError(f"{name} must be {list(like.shape)}, got {tuple(shape)}")
    if not (0 < h <= _INT32_MAX and 0 < d <= _INT32_MAX):
        raise ValueError(f"{name} is {tuple(shape)}")
    if t.is_contiguous():
        return h * d, d
    ld, hs, inner = t.stride()
    ld, hs = ld if n > 1 else h * d, hs if h > 1 else d
    apart = hs >= d and ld >= (h - 1) * hs + d or ld >= d and hs >= (n - 1) * ld + d  # rows of heads, or heads of rows
    if n > 0 and (d > 1 and inner != 1 or h > 1 and n > 1 and not apart or min(ld, hs) < d):
        raise ValueError(f"{name}: a head's columns must be next to each other, heads and rows must not overlap, "
                         f"got strides {t.stride()}")
    return ld, hs


def rotary_frequencies(dim: int, axes: int = 1, base: float = 10000.0, scaling: Optional[str] = None,
                       factor: float = 1.0, length: int = 4096, low: float = 1.0, high: float = 32.0,
                       device=None) -> torch.Tensor:
    """Radians per position, [F] fp64, of ``dim`` = 2 axes F rotated columns:
    ``base ** (-f / F)``. For positions ``factor`` times as far as those a model
    learned (``length`` of them), ``scaling`` stretches them: "linear" divides all
    frequencies by ``factor``; "base" raises the base so that the slowest pair's
    is; "parts" divides those of pairs that make fewer than ``low`` turns over
    ``length``, keeps those of more than ``high``, and blends in between."""
    dim, axes = int(dim), int(axes)
    if axes < 1 or dim < 2 or dim % (2 * axes):
        raise ValueError(f"{dim} columns are not pairs for {axes} axes")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError(f"base = {base}, factor = {factor}")
    pairs = dim // (2 * axes)
    if scaling == "base":
        base = base * factor ** (pairs / max(1, pairs - 1))
    f = base ** -(torch.arange(pairs, dtype=torch.float64) / pairs)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not high > low:
            raise ValueError(f"low = {low}, high = {high}")
        keep = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    elif scaling not in (None, "none", "base"):
        raise ValueError(f"scaling must be 'linear', 'base' or 'parts', got {scaling!r}")
    return f.to(device) if device is not None else f


def rotary(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool = False,
           inverse: bool = False, amplitude: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Turns the pairs of the first ``2 axes F`` columns of each head of ``x``
    ([N,H,D] fp16, bf16 or fp32, rows of heads or heads of rows, of a wider tensor as
    well) by ``position *
    freq`` and copies the others. ``positions`` int32 [N], or [N,axes] (up to 4
    axes; a slice of sites' coordinates is fine), ``freqs`` fp64 [F] in radians
    (:func:`rotary_frequencies`): pair ``p = axis F + f``, columns (2p, 2p + 1) where
    ``interleaved``, else (p, axes F + p). ``inverse`` turns back, which is the
    gradient; ``amplitude`` scales what is turned. ``out`` may be x itself, but not
    overlap it otherwise."""
    ldx, hx = _heads(x, "x", _NORM_DTYPES)
    n, h, d = x.shape
    dev = x.device
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a tensor")
    if positions.dtype != torch.int32:
        raise TypeError(f"positions must be {torch.int32}, got {positions.dtype}")
    if positions.device != dev:
        raise ValueError(f"positions is on {positions.device}, not on {dev}")
    if positions.dim() not in (1, 2) or positions.shape[0] != n or positions.dim() == 2 and not 1 <= positions.shape[1] <= 4:
        raise ValueError(f"positions must be [{n}] or [{n},axes] with 1 to 4 axes, got {tuple(positions.shape)}")
    axes = positions.shape[1] if positions.dim() == 2 else 1
    ap = positions.stride(1) if positions.dim() == 2 else 1
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a tensor [F]")
    _dense(freqs, "freqs", torch.float64, tuple(freqs.shape), dev)
    f = freqs.shape[0]
    if f < 1 or 2 * axes * f > d:
        raise ValueError(f"{axes} axes of {f} pairs do not fit {d} columns")
    if out is None:
        out, ldo, ho = x.new_empty((n, h, d)), h * d, d
    else:
        ldo, ho = _heads(out, "out", (x.dtype,), x)
        torch.autograd.graph.increment_version(out)  # a change in place, for autograd's checks
    _call(dev, "submconv_rotary", _ptr(x), ldx, hx, n, h, d, _ptr(positions), positions.stride(0), ap, axes,
          _ptr(freqs), f, int(bool(interleaved)), int(bool(inverse)), amplitude, _ptr(out), ldo, ho,
          _NORM_DTYPES[x.dtype])
    return out


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


def _attention_args(q, k, v, offsets, k_offsets, k_lengths, scale):
    """Checks shared by both directions: the C arguments from q on, without the
    results, and the sizes (nq, nk, heads, key heads, columns, items)."""
    ldq, hq = _heads(q, "q", _DTYPES)
    ldk, hk = _heads(k, "k", (q.dtype,))
    ldv, hv = _heads(v, "v", (q.dtype,), k)
    nq, heads, d = q.shape
    nk, kv_heads, dk = k.shape
    dev = q.device
    if k.device != dev:
        raise ValueError(f"k is on {k.device}, not on {dev}")
    if dk != d:
        raise ValueError(f"q has {d} columns a head, k has {dk}")
    if heads % kv_heads:
        raise ValueError(f"{heads} query heads do not share {kv_heads} key heads")
    items = _items(offsets, "offsets", dev)
    if k_offsets is None:
        if nk != nq and offsets is not None:
            raise ValueError(f"{nq} queries and {nk} keys: k_offsets are needed")
        k_offsets = offsets
    elif _items(k_offsets, "k_offsets", dev) != items:
        raise ValueError(f"{items} items of queries, {k_offsets.shape[0] - 1} of keys")
    _optional(k_lengths, "k_lengths", torch.int32, (items,), dev)
    if scale is None:
        scale = d ** -0.5
    args = (_ptr(q), ldq, hq, nq, _ptr(k), ldk, hk, _ptr(v), ldv, hv, nk, heads, kv_heads, d, _ptr(offsets),
            _ptr(k_offsets), _ptr(k_lengths), items, scale)
    return args, (nq, nk, heads, kv_heads, d, items)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: Optional[torch.Tensor] = None,
              k_offsets: Optional[torch.Tensor] = None, k_lengths: Optional[torch.Tensor] = None,
              causal: bool = False, scale: Optional[float] = None, return_lse: bool = False):
    """Attention of each item's queries over its keys: ``softmax(scale q k^T) v`` in
    q's dtype (fp16 or bf16). ``q`` [Nq,Hq,D], ``k`` and ``v`` [Nk,Hk,D], slices of
    a projection for example: D a multiple of 8 up to 128, starts on 16 bytes,
    strides in multiples of 8; Hq is a multiple of Hk, neighbouring query heads
    share a key head.

    ``offsets`` are the queries' items, ``k_offsets`` the keys' (None: the same, or
    with no offsets either one item of all queries and all keys),
    ``k_lengths`` [items] int32 how many of an item's keys are there (None: all; a
    cache with room). ``causal``: the last query of an item sees all of its keys,
    each earlier one a key less; the keys and values that a query does not see
    have to be finite all the same. So one new token per item over its cache is
    ``offsets = 0 .. items``. ``scale`` defaults to ``D ** -0.5``. A query without
    keys gives zeros. ``return_lse``: also the fp32 ``log sum exp`` of the scores
    [Nq,Hq] that :func:`attention_backward` takes (-inf without keys)."""
    args, (nq, nk, heads, kv_heads, d, items) = _attention_args(q, k, v, offsets, k_offsets, k_lengths, scale)
    out = q.new_empty((nq, heads, d))
    lse = q.new_empty((nq, heads), dtype=torch.float32) if return_lse else None
    ws, nb = _workspace("submconv_attention_workspace_bytes", q, nq, nk, heads, kv_heads, d, items, int(bool(causal)))
    _call(q.device, "submconv_attention", *args, int(bool(causal)), _ptr(out), _ptr(lse), _DTYPES[q.dtype], _ptr(ws),
          nb)
    return (out, lse) if return_lse else out


def attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                       k_offsets: Optional[torch.Tensor] = None, k_lengths: Optional[torch.Tensor] = None,
                       causal: bool = False, scale: Optional[float] = None, needs=(True, True, True)):
    """``(grad_q, grad_k, grad_v)`` of :func:`attention` in q's dtype; ``out`` and
    ``lse`` as it returned them. ``needs`` leaves gradients out (None)."""
    args, (nq, nk, heads, kv_heads, d, items) = _attention_args(q, k, v, offsets, k_offsets, k_lengths, scale)
    ldg, hg = _heads(grad_out, "grad_out", (q.dtype,), q)
    _dense(out, "out", q.dtype, (nq, heads, d), q.device)
    _dense(lse, "lse", torch.float32, (nq, heads), q.device)
    gq = q.new_empty((nq, heads, d)) if needs[0] else None
    gk = q.new_empty((nk, kv_heads, d)) if needs[1] else None
    gv = q.new_empty((nk, kv_heads, d)) if needs[2] else None
    ws, nb = _workspace("submconv_attention_backward_workspace_bytes", q, nq, nk, heads, kv_heads, d, items,
                        int(bool(causal)))
    _call(q.device, "submconv_attention_backward", _ptr(grad_out), ldg, hg, _ptr(out), _ptr(lse), *args,
          int(bool(causal)), _ptr(gq), _ptr(gk), _ptr(gv), _DTYPES[q.dtype], _ptr(ws), nb)
    return gq, gk, gv


# ---------------------------------------------------------------------------
# autograd and modules
# ---------------------------------------------------------------------------


class GroupNormFunction(torch.autograd.Function):
    """Autograd over :func:`group_norm`."""

    @staticmethod
    def forward(ctx, x, weight, bias, groups, eps, act, offsets):
        y, mean, rstd = group_norm(x, groups, weight, bias, eps, act, offsets, return_stats=True)
        ctx.save_for_backward(x, weight, bias, mean, rstd, offsets)
        ctx.act = act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, weight, bias, mean, rstd, offsets = ctx.saved_tensors
        grads = group_norm_backward(grad_out.contiguous(), x, mean, rstd, weight, bias, ctx.act, offsets,
                                    ctx.needs_input_grad[:3])
        return (*grads, None, None, None, None)


class RotaryFunction(torch.autograd.Function):
    """Autograd over :func:`rotary`, for the rows."""

    @staticmethod
    def forward(ctx, x, positions, freqs, interleaved, amplitude):
        ctx.save_for_backward(positions, freqs)
        ctx.how = interleaved, amplitude
        return rotary(x, positions, freqs, interleaved, False, amplitude)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        positions, freqs = ctx.saved_tensors
        interleaved, amplitude = ctx.how
        return rotary(grad_out.contiguous(), positions, freqs, interleaved, True, amplitude), None, None, None, None


class AttentionFunction(torch.autograd.Function):
    """Autograd over :func:`attention`, for queries, keys and values."""

    @staticmethod
    def forward(ctx, q, k, v, offsets, k_offsets, k_lengths, causal, scale):
        out, lse = attention(q, k, v, offsets, k_offsets, k_lengths, causal, scale, return_lse=True)
        ctx.save_for_backward(q, k, v, out, lse, offsets, k_offsets, k_lengths)
        ctx.how = causal, scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        grad_out = grad_out.contiguous()
        if grad_out.data_ptr() % 16:  # a piece of a tensor that autograd took apart
            grad_out = grad_out.clone()
        grads = attention_backward(grad_out, *ctx.saved_tensors, *ctx.how, ctx.needs_input_grad[:3])
        return (*grads, None, None, None, None, None)


class GroupNorm(torch.nn.Module):
    """Group norm over ``channels`` in ``groups`` with fp32 weight and bias and an
    activation."""

    def __init__(self, groups: int, channels: int, eps: float = 1e-5, act: Optional[str] = None, device=None):
        super().__init__()
        _groups(groups, channels)
        _act(act)
        self.groups, self.eps, self.act = groups, eps, act
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(channels, device=device))

    def forward(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
        if _recorded(x, self.weight, self.bias):
            return GroupNormFunction.apply(x, self.weight, self.bias, self.groups, self.eps, self.act, offsets)
        return group_norm(x, self.groups, self.weight, self.bias, self.eps, self.act, offsets)


class SparseAttention(torch.nn.Module):
    """Attention with its projections on the rows of packed items: among an item's
    rows, or, with ``context`` (its row width), over an item's rows of another
    tensor. ``channels`` is the row width, ``heads`` of ``dim`` columns (default
    channels / heads), ``kv_heads`` (default heads) of keys and values. With
    ``rotary`` columns of a head and ``axes`` coordinates, queries and keys are
    turned by their rows' positions [N,axes] (not over a context)."""

    def __init__(self, channels: int, heads: int, dim: Optional[int] = None, kv_heads: Optional[int] = None,
                 context: Optional[int] = None, rotary: int = 0, axes: int = 3, causal: bool = False,
                 interleaved: bool = True, device=None, dtype=torch.float16):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        if heads < 1 or kv_heads < 1 or heads % kv_heads:
            raise ValueError(f"{heads} query heads do not share {kv_heads} key heads")
        if dim is None:
            if channels % heads:
                raise ValueError(f"{channels} channels do not make {heads} heads")
            dim = channels // heads
        if dim < 8 or dim > 128 or dim % 8:
            raise ValueError(f"{dim} columns a head: multiples of 8 up to 128 are supported")
        if rotary > dim or rotary and context is not None:
            raise ValueError(f"{rotary} of {dim} columns turn" + (" over a context" if context is not None else ""))
        self.heads, self.kv_heads, self.dim, self.causal, self.interleaved = heads, kv_heads, dim, causal, interleaved
        self.own, self.rotary, self.axes = context is None, rotary, axes
        if self.own:
            self.proj_in = Linear(channels, (heads + 2 * kv_heads) * dim, device=device, dtype=dtype)
        else:
            self.proj_in = Linear(channels, heads * dim, device=device, dtype=dtype)
            self.proj_context = Linear(context, 2 * kv_heads * dim, device=device, dtype=dtype)
        self.proj_out = Linear(heads * dim, channels, device=device, dtype=dtype)
        self.register_buffer("freqs", rotary_frequencies(rotary, axes, device=device) if rotary else None)

    def _apply(self, fn, recurse=True):
        freqs = self.freqs
        super()._apply(fn, recurse)
        if freqs is not None:  # moves with the module, and stays in 64 bits whatever its type
            if freqs.is_meta and not self.freqs.is_meta:  # it has memory now, but no values
                freqs = rotary_frequencies(self.rotary, self.axes, device="cpu")
            self.freqs = freqs.to(self.freqs.device)
        return self

    def forward(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                positions: Optional[torch.Tensor] = None, context: Optional[torch.Tensor] = None,
                context_offsets: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        if self.own and not (context is None and context_offsets is None):
            raise ValueError("the module attends among an item's rows: it has no use for a context")
        if self.freqs is not None:
            if positions is None:
                raise ValueError("positions are needed to turn queries and keys")
            if not isinstance(positions, torch.Tensor):
                raise TypeError("positions must be a tensor")
            if positions.dim() not in (1, 2) or (positions.shape[1] if positions.dim() == 2 else 1) != self.axes:
                raise ValueError(f"positions must be [N,{self.axes}], the module's axes, got {tuple(positions.shape)}")
        h, hk, d = self.heads, self.kv_heads, self.dim
        rows = self.proj_in(x).view(x.shape[0], h + 2 * hk if self.own else h, d)
        if self.own:
            both, v = rows.split([h + hk, hk], 1)
            if self.freqs is not None:
                if _recorded(both):
                    both = RotaryFunction.apply(both, positions, self.freqs, self.interleaved, 1.0)
                else:
                    rotary(both, positions, self.freqs, self.interleaved, out=both)
            q, k = both.split([h, hk], 1)
        else:
            if context is None:
                raise ValueError("a context is needed")
            q = rows
            k, v = self.proj_context(context).view(context.shape[0], 2 * hk, d).split([hk, hk], 1)
            if context_offsets is None and offsets is not None:
                raise ValueError("context_offsets are needed")
        if _recorded(q, k, v):
            out = AttentionFunction.apply(q, k, v, offsets, context_offsets, None, self.causal, None)
        else:
            out = attention(q, k, v, offsets, context_offsets, None, self.causal)
        return self.proj_out(out.view(x.shape[0], h * d), residual=residual)
