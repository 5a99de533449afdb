"""Dense layers on site features: layer norm, linear with a fused epilogue and
the gated feed-forward block, forward and backward, on the library's kernels.

Rows are sites; ``x``, ``grad_out`` and ``residual`` may be rows of a wider
tensor (any row stride, columns next to each other). The matrix layers take
fp16 or bf16 with fp32 biases and weights ``[Cin, Cout]`` (a 1x1x1
convolution's ``W[0]``); layer norm takes fp32 as well.

The functions compute without recording gradients; the ``*Function`` classes
and the modules are the autograd form.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _DTYPES, _check, load_library

__all__ = [
    "layer_norm", "layer_norm_backward", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward",
    "LayerNormFunction", "LinearFunction", "GatedFeedForwardFunction", "LayerNorm", "Linear",
    "GatedFeedForward", "ACTIVATIONS",
]

#: names of the activations, as SUBMCONV_ACT_*
ACTIVATIONS = {"none": 0, None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_NORM_DTYPES = {**_DTYPES, torch.float32: 2}
_INT32_MAX = 2 ** 31 - 1  # widths cross the C ABI as int32, which would cut larger ones


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


try:
    from torch._C import _cuda_getCurrentRawStream as _current_stream
except ImportError:  # a torch without it: the same through the public object

    def _current_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _call(device: torch.device, name: str, *args) -> None:
    """Calls an entry point on the device's current stream, its last argument."""
    fn = getattr(load_library(), name)
    if device.index == torch.cuda.current_device():
        status = fn(*args, _current_stream(device.index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(device.index))
    if status:
        _check(status)


def _act(act) -> int:
    try:
        return ACTIVATIONS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {[a for a in ACTIVATIONS if a]}, got {act!r}") from None


def _rows(t, name: str, dtypes, cols: Optional[int] = None, like=None) -> int:
    """Checks a matrix of rows and returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    n, c = t.shape
    if c > _INT32_MAX:
        raise ValueError(f"{name} has {c} columns")
    if cols is not None and c != cols:
        raise ValueError(f"{name} must have {cols} columns, got {tuple(t.shape)}")
    if like is not None:
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")
        if n != like.shape[0]:
            raise ValueError(f"{name} must have {like.shape[0]} rows, got {tuple(t.shape)}")
    ld, inner = t.stride()
    if n > 1 and ld < c or c > 1 and inner != 1 and n > 0:
        raise ValueError(f"{name}: columns must be next to each other and rows must not overlap, "
                         f"got strides {t.stride()}")
    return ld if n > 1 else c


def _dense(t, name: str, dtype, shape: Tuple[int, ...], device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _optional(t, name: str, dtype, shape, device) -> None:
    if t is not None:
        _dense(t, name, dtype, shape, device)


def _matrix(t, name: str, x) -> Tuple[int, int]:
    """Checks a weight matrix of x's type and returns its shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {tuple(t.shape)}")
    shape = tuple(t.shape)
    if max(shape) > _INT32_MAX:
        raise ValueError(f"{name} is {shape}")
    _dense(t, name, x.dtype, shape, x.device)
    return shape


def _aligned(*parts) -> int:
    """Whether every (tensor, row stride) starts on 16 bytes with rows of
    16-byte multiples."""
    return int(all(t is None or (t.data_ptr() % 16 == 0 and ld % 8 == 0) for t, ld in parts))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(query: str, *sizes: int) -> int:
    v = int(getattr(load_library(), query)(*sizes))
    if v < 0:
        _check(v)
    return v


def _workspace(query: str, x: torch.Tensor, *sizes: int):
    """(tensor or None, bytes) of an operator's workspace."""
    need = _workspace_bytes(query, *sizes)
    return (x.new_empty((need,), dtype=torch.uint8) if need else None), need


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, return_stats: bool = False):
    """Layer norm over the columns of ``x`` ([N,C] fp16, bf16 or fp32; C up to
    8192) with fp32 ``weight`` and ``bias`` ([C], either may be None):
    ``y`` in x's dtype, or ``(y, mean, rstd)`` with the fp32 row statistics
    that :func:`layer_norm_backward` takes."""
    ld = _rows(x, "x", _NORM_DTYPES)
    n, c = x.shape
    dev = x.device
    _optional(weight, "weight", torch.float32, (c,), dev)
    _optional(bias, "bias", torch.float32, (c,), dev)
    y = x.new_empty((n, c))
    mean = rstd = None
    if return_stats:
        mean = x.new_empty((n,), dtype=torch.float32)
        rstd = x.new_empty((n,), dtype=torch.float32)
    _call(dev, "submconv_layer_norm", _ptr(x), ld, n, c, _ptr(weight), _ptr(bias), eps, _ptr(y), _ptr(mean),
          _ptr(rstd), _NORM_DTYPES[x.dtype])
    return (y, mean, rstd) if return_stats else y


def layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, needs=(True, True, True)):
    """``(grad_x, grad_weight, grad_bias)`` of :func:`layer_norm`: grad_x in
    x's dtype, the others fp32 [C]. ``needs`` leaves gradients out (None)."""
    ldx = _rows(x, "x", _NORM_DTYPES)
    n, c = x.shape
    dev = x.device
    ldg = _rows(grad_out, "grad_out", (x.dtype,), c, x)
    _dense(mean, "mean", torch.float32, (n,), dev)
    _dense(rstd, "rstd", torch.float32, (n,), dev)
    _optional(weight, "weight", torch.float32, (c,), dev)
    gx = x.new_empty((n, c)) if needs[0] else None
    gw = x.new_empty((c,), dtype=torch.float32) if needs[1] else None
    gb = x.new_empty((c,), dtype=torch.float32) if needs[2] else None
    ws, nb = None, 0
    if needs[1] or needs[2]:
        ws, nb = _workspace("submconv_layer_norm_backward_workspace_bytes", x, n, c)
    _call(dev, "submconv_layer_norm_backward", _ptr(grad_out), ldg, _ptr(x), ldx, n, c, _ptr(mean),
          _ptr(rstd), _ptr(weight), _ptr(gx), _ptr(gw), _ptr(gb), _NORM_DTYPES[x.dtype], _ptr(ws), nb)
    return gx, gw, gb


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------


def linear(x: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None, act: Optional[str] = None,
           residual: Optional[torch.Tensor] = None, return_pre: bool = False):
    """``act(x W + bias) + residual`` in x's dtype (fp16 or bf16): x [N,Cin],
    W [Cin,Cout], bias fp32 [Cout], residual [N,Cout]; ``act`` one of
    :data:`ACTIVATIONS`. ``return_pre``: also ``x W + bias``, which
    :func:`linear_backward` takes."""
    ldx = _rows(x, "x", _DTYPES)
    n, cin = x.shape
    dev = x.device
    k, cout = _matrix(W, "W", x)
    if k != cin:
        raise ValueError(f"W is {tuple(W.shape)} but x has Cin = {cin}")
    _optional(bias, "bias", torch.float32, (cout,), dev)
    a = _act(act)
    ldr = _rows(residual, "residual", (x.dtype,), cout, x) if residual is not None else 0
    out = x.new_empty((n, cout))
    pre = x.new_empty((n, cout)) if return_pre else None
    ws, nb = _workspace("submconv_linear_workspace_bytes", x, n, cin, cout, _aligned((x, ldx), (W, cout)))
    _call(dev, "submconv_linear", _ptr(x), ldx, n, _ptr(W), _ptr(bias), _ptr(residual), ldr, _ptr(out),
          _ptr(pre), cin, cout, a, _DTYPES[x.dtype], _ptr(ws), nb)
    return (out, pre) if return_pre else out


def linear_backward(grad_out: torch.Tensor, x: torch.Tensor, W: torch.Tensor, pre: Optional[torch.Tensor] = None,
                    act: Optional[str] = None, needs=(True, True, True)):
    """``(grad_x, grad_W, grad_bias)`` of :func:`linear`: the first two in x's
    dtype, the last fp32. ``pre`` as the forward returned it (not needed
    without an activation). The residual's gradient is ``grad_out`` itself.
    ``needs`` leaves gradients out (None)."""
    ldx = _rows(x, "x", _DTYPES)
    n, cin = x.shape
    dev = x.device
    k, cout = _matrix(W, "W", x)
    if k != cin:
        raise ValueError(f"W is {tuple(W.shape)} but x has Cin = {cin}")
    ldg = _rows(grad_out, "grad_out", (x.dtype,), cout, x)
    a = _act(act)
    if a:
        _dense(pre, "pre", x.dtype, (n, cout), dev)
    gx = x.new_empty((n, cin)) if needs[0] else None
    gw = x.new_empty((cin, cout)) if needs[1] else None
    gb = x.new_empty((cout,), dtype=torch.float32) if needs[2] else None
    ws, nb = _workspace("submconv_linear_backward_workspace_bytes", x, n, cin, cout, a,
                        _aligned((x, ldx), (W, cout), (grad_out, ldg)))
    _call(dev, "submconv_linear_backward", _ptr(grad_out), ldg, n, _ptr(x), ldx, _ptr(W), _ptr(pre) if a else
          None, _ptr(gx), _ptr(gw), _ptr(gb), cin, cout, a, _DTYPES[x.dtype], _ptr(ws), nb)
    return gx, gw, gb


# ---------------------------------------------------------------------------
# gated feed-forward
# ---------------------------------------------------------------------------


def _ffn_shapes(x, W_in, W_out):
    cin = x.shape[1]
    k, two = _matrix(W_in, "W_in", x)
    hidden, cout = _matrix(W_out, "W_out", x)
    if k != cin or two != 2 * hidden:
        raise ValueError(f"W_in is {tuple(W_in.shape)}, W_out {tuple(W_out.shape)}: W_in must be "
                         f"[Cin,2*hidden] = [{cin},{2 * hidden}]")
    return cin, hidden, cout


def gated_ffn(x: torch.Tensor, W_in: torch.Tensor, b_in: Optional[torch.Tensor], W_out: torch.Tensor,
              b_out: Optional[torch.Tensor] = None, act: str = "silu", residual: Optional[torch.Tensor] = None,
              return_pre: bool = False):
    """``(act(g) * u) W_out + b_out + residual`` with ``[g | u] = x W_in +
    b_in`` in x's dtype (fp16 or bf16): x [N,Cin], W_in [Cin,2*hidden] (gate
    columns first), W_out [hidden,Cout], fp32 biases. ``return_pre``: also
    ``[g | u]``, which :func:`gated_ffn_backward` takes. From 9 rows on ``act(g)
    * u`` is rounded to x's dtype between the products (past 65504 it is infinite
    in fp16); up to 8 rows it stays fp32."""
    ldx = _rows(x, "x", _DTYPES)
    n = x.shape[0]
    dev = x.device
    cin, hidden, cout = _ffn_shapes(x, W_in, W_out)
    _optional(b_in, "b_in", torch.float32, (2 * hidden,), dev)
    _optional(b_out, "b_out", torch.float32, (cout,), dev)
    a = _act(act)
    ldr = _rows(residual, "residual", (x.dtype,), cout, x) if residual is not None else 0
    out = x.new_empty((n, cout))
    pre = x.new_empty((n, 2 * hidden)) if return_pre else None
    query = "submconv_gated_ffn_workspace_bytes" if return_pre else "submconv_gated_ffn_inference_workspace_bytes"
    ws, nb = _workspace(query, x, n, cin, hidden, cout,
                        _aligned((x, ldx), (W_in, 2 * hidden), (W_out, cout)))
    _call(dev, "submconv_gated_ffn", _ptr(x), ldx, n, _ptr(W_in), _ptr(b_in), _ptr(W_out), _ptr(b_out),
          _ptr(residual), ldr, _ptr(out), _ptr(pre), cin, hidden, cout, a, _DTYPES[x.dtype], _ptr(ws), nb)
    return (out, pre) if return_pre else out


def gated_ffn_backward(grad_out: torch.Tensor, x: torch.Tensor, W_in: torch.Tensor, W_out: torch.Tensor,
                       pre: torch.Tensor, act: str = "silu", needs=(True, True, True, True, True)):
    """``(grad_x, grad_W_in, grad_b_in, grad_W_out, grad_b_out)`` of
    :func:`gated_ffn`: matrices in x's dtype, biases fp32. ``pre`` as the
    forward returned it. The residual's gradient is ``grad_out`` itself.
    ``needs`` leaves gradients out (None)."""
    ldx = _rows(x, "x", _DTYPES)
    n = x.shape[0]
    dev = x.device
    cin, hidden, cout = _ffn_shapes(x, W_in, W_out)
    ldg = _rows(grad_out, "grad_out", (x.dtype,), cout, x)
    _dense(pre, "pre", x.dtype, (n, 2 * hidden), dev)
    a = _act(act)
    shapes = [((n, cin), x.dtype), ((cin, 2 * hidden), x.dtype), ((2 * hidden,), torch.float32),
              ((hidden, cout), x.dtype), ((cout,), torch.float32)]
    g = [x.new_empty(s, dtype=d) if need else None for (s, d), need in zip(shapes, needs)]
    ws, nb = _workspace("submconv_gated_ffn_backward_workspace_bytes", x, n, cin, hidden, cout,
                        _aligned((x, ldx), (W_in, 2 * hidden), (W_out, cout), (grad_out, ldg)))
    _call(dev, "submconv_gated_ffn_backward", _ptr(grad_out), ldg, n, _ptr(x), ldx, _ptr(W_in), _ptr(W_out),
          _ptr(pre), _ptr(g[0]), _ptr(g[1]), _ptr(g[2]), _ptr(g[3]), _ptr(g[4]), cin, hidden, cout, a,
          _DTYPES[x.dtype], _ptr(ws), nb)
    return tuple(g)


# ---------------------------------------------------------------------------
# autograd and modules
# ---------------------------------------------------------------------------


class LayerNormFunction(torch.autograd.Function):
    """Autograd over :func:`layer_norm`."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm(x, weight, bias, eps, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, weight, mean, rstd = ctx.saved_tensors
        gx, gw, gb = layer_norm_backward(grad_out.contiguous(), x, mean, rstd, weight, ctx.needs_input_grad[:3])
        return gx, gw, gb, None


class LinearFunction(torch.autograd.Function):
    """Autograd over :func:`linear`; keeps the pre-activation only where there
    is an activation."""

    @staticmethod
    def forward(ctx, x, W, bias, residual, act):
        pre = None
        if _act(act):
            out, pre = linear(x, W, bias, act, residual, return_pre=True)
        else:
            out = linear(x, W, bias, act, residual)
        ctx.save_for_backward(x, W, pre)
        ctx.act = act
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, W, pre = ctx.saved_tensors
        g = grad_out.contiguous()
        gx, gw, gb = linear_backward(g, x, W, pre, ctx.act, ctx.needs_input_grad[:3])
        return gx, gw, gb, g if ctx.needs_input_grad[3] else None, None


class GatedFeedForwardFunction(torch.autograd.Function):
    """Autograd over :func:`gated_ffn`."""

    @staticmethod
    def forward(ctx, x, W_in, b_in, W_out, b_out, residual, act):
        out, pre = gated_ffn(x, W_in, b_in, W_out, b_out, act, residual, return_pre=True)
        ctx.save_for_backward(x, W_in, W_out, pre)
        ctx.act = act
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x, W_in, W_out, pre = ctx.saved_tensors
        g = grad_out.contiguous()
        grads = gated_ffn_backward(g, x, W_in, W_out, pre, ctx.act, ctx.needs_input_grad[:5])
        return (*grads, g if ctx.needs_input_grad[5] else None, None)


def _recorded(*tensors: Optional[torch.Tensor]) -> bool:
    """Whether autograd will ask for a gradient of any of them: only then do the
    modules take the functions that keep what the backward pass reads."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


class LayerNorm(torch.nn.Module):
    """Layer norm over ``channels`` with fp32 weight and bias."""

    def __init__(self, channels: int, eps: float = 1e-5, device=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(channels, device=device))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if _recorded(x, self.weight, self.bias):
            return LayerNormFunction.apply(x, self.weight, self.bias, self.eps)
        return layer_norm(x, self.weight, self.bias, self.eps)


def _init_matrix(rows: int, cols: int, device, dtype) -> torch.nn.Parameter:
    return torch.nn.Parameter((torch.randn(rows, cols, device=device) * rows ** -0.5).to(dtype))


class Linear(torch.nn.Module):
    """``act(x W + b) + residual`` with W [Cin,Cout] of ``dtype`` and an fp32
    bias."""

    def __init__(self, cin: int, cout: int, bias: bool = True, act: Optional[str] = None, device=None,
                 dtype=torch.float16):
        super().__init__()
        _act(act)
        self.act = act
        self.weight = _init_matrix(cin, cout, device, dtype)
        self.bias = torch.nn.Parameter(torch.zeros(cout, device=device)) if bias else None

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        if _recorded(x, self.weight, self.bias, residual):
            return LinearFunction.apply(x, self.weight, self.bias, residual, self.act)
        return linear(x, self.weight, self.bias, self.act, residual)


class GatedFeedForward(torch.nn.Module):
    """Gated feed-forward block ``(act(g) * u) W_out + b_out + residual``."""

    def __init__(self, channels: int, hidden: int, act: str = "silu", bias: bool = True, device=None,
                 dtype=torch.float16):
        super().__init__()
        _act(act)
        self.act = act
        self.w_in = _init_matrix(channels, 2 * hidden, device, dtype)
        self.w_out = _init_matrix(hidden, channels, device, dtype)
        self.b_in = torch.nn.Parameter(torch.zeros(2 * hidden, device=device)) if bias else None
        self.b_out = torch.nn.Parameter(torch.zeros(channels, device=device)) if bias else None

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        if _recorded(x, self.w_in, self.b_in, self.w_out, self.b_out, residual):
            return GatedFeedForwardFunction.apply(x, self.w_in, self.b_in, self.w_out, self.b_out, residual, self.act)
        return gated_ffn(x, self.w_in, self.b_in, self.w_out, self.b_out, self.act, residual)
