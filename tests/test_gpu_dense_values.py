"""Values of the dense layers where fp32 formulas lose digits or range: the
negative tail of the erf form of gelu, in bf16 which can hold it, bf16's
largest numbers, widths that 32 bits do not hold, and hidden values past fp16."""
import numpy as np
import pytest
import torch
from scipy.special import ndtr

gpu = pytest.mark.gpu
V = 2.0 ** -24
UB = 2.0 ** -8  # unit roundoff of bf16


def _sc():
    import submanifold_sparse_convolution_hash_amd as sc
    sc.load_library()
    return sc


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _eye(c, dev):
    return torch.eye(c, dtype=torch.bfloat16, device=dev)


def _check(got, ref, tol, what):
    err = np.abs(_np(got) - ref)
    assert (err <= tol).all(), (what, float(np.nanmax(err / tol)), int((~(err <= tol)).sum()))


@gpu
@pytest.mark.parametrize("n", [8, 200])
def test_gelu_tail(dev, n):
    """gelu = z Phi(z) and its slope Phi(z) + z phi(z) for z from 0 to -12, to a
    bf16's own rounding. An identity weight hands z on exactly. Phi is half of
    erfc(-z / sqrt 2), whose argument is off by 2 v: (z^2 + 1) 2 v of its value, next
    to erfc's own 16 ulps (32 v) and three products; phi is exp of an argument off
    by 1.5 v z^2 and a few ulps more."""
    sc = _sc()
    c = 32
    x = torch.linspace(-12, 0, n * c).reshape(n, c).to(torch.bfloat16).to(dev)
    z = _np(x)
    big, pdf = ndtr(z), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    rel = V * (2 * z * z + 40)
    value, slope = z * big, big + z * pdf
    tol_v = (rel + UB) * np.abs(value) + 1e-38
    tol_s = rel * (big + np.abs(z) * pdf) + UB * np.abs(slope) + 1e-38
    eye = _eye(c, dev)
    _check(sc.linear(x, eye, act="gelu"), value, tol_v, "linear")
    # the gated block with u = 1 on its gate's side
    Wi = torch.cat([eye, torch.zeros_like(eye)], 1).contiguous()
    bi = torch.cat([torch.zeros(c), torch.ones(c)]).to(dev)
    _check(sc.gated_ffn(x, Wi, bi, eye, act="gelu"), value, tol_v, "gated")
    out, pre = sc.gated_ffn(x, Wi, bi, eye, act="gelu", return_pre=True)
    _check(out, value, tol_v, "gated with pre")
    one = torch.ones_like(x)
    _check(sc.linear_backward(one, x, eye, x, act="gelu")[0], slope, tol_s, "slope")
    _check(sc.gated_ffn_backward(one, x, Wi, eye, pre, act="gelu")[0], slope, tol_s, "gated slope")
    # h, formed again from pre, against one row of ones at a time
    dy = torch.zeros((n, c), dtype=torch.bfloat16, device=dev)
    dy[n // 2] = 1
    gw = sc.gated_ffn_backward(dy, x, Wi, eye, pre, act="gelu")[3]
    _check(gw, np.repeat(value[n // 2][:, None], c, 1), np.repeat(tol_v[n // 2][:, None], c, 1), "h of the gradient")


@gpu
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n", [8, 64])
def test_activations_of_huge_values(dev, n, act):
    """Up to bf16's largest numbers the value is z or 0 and the slope 1 or 0."""
    sc = _sc()
    c = 16
    big = torch.tensor([1e9, 1e13, 2e19, 1e25, 1e30, 3e38])
    x = torch.cat([big, -big]).repeat(n * c // 12 + 1)[:n * c].reshape(n, c).to(torch.bfloat16).to(dev)
    eye = _eye(c, dev)
    ref, on = (x, torch.ones_like(x)) if act == "none" else (x.clamp(min=0), (x > 0).to(x.dtype))
    assert torch.equal(sc.linear(x, eye, act=act), ref)
    one = torch.ones_like(x)
    gx, _, gb = sc.linear_backward(one, x, eye, x, act=act)
    assert torch.equal(gx, on)
    assert torch.equal(gb, on.float().sum(0))
    pre = torch.cat([x, one], 1).contiguous()
    Wi = torch.cat([eye, torch.zeros_like(eye)], 1).contiguous()
    assert torch.equal(sc.gated_ffn_backward(one, x, Wi, eye, pre, act=act)[0], on)


@gpu
def test_more_columns_than_32_bits_are_refused(dev):
    """Sizes past 2^31 do not reach the library cut to 32 bits."""
    sc = _sc()
    many = 2 ** 32 + 8
    h = dict(dtype=torch.float16, device=dev)
    wide, tall = torch.empty((1, many), **h), torch.empty((many, 1), **h)
    one = torch.zeros((1, 1), **h)
    stat = torch.zeros(1, device=dev)
    for call in (lambda: sc.layer_norm(wide), lambda: sc.layer_norm_backward(wide, wide, stat, stat),
                 lambda: sc.linear(wide, tall), lambda: sc.linear(one, wide),
                 lambda: sc.linear_backward(wide, one, wide),
                 lambda: sc.gated_ffn(one, torch.empty((1, 2 * many), **h), None, tall)):
        with pytest.raises(ValueError):
            call()


@gpu
def test_range_of_the_hidden_rows(dev):
    """Hidden values of 90000, which fp16 does not hold: up to 8 rows they stay fp32,
    from 9 rows on they are operands of the data's type, as documented; bf16 holds
    them (90000 to one rounding) at any count."""
    sc = _sc()
    c = 16
    for dtype, n, ref in ((torch.float16, 8, 90000 / 64), (torch.float16, 9, float("inf")),
                          (torch.bfloat16, 8, 90000 / 64), (torch.bfloat16, 9, 90000 / 64)):
        x = torch.full((n, c), 300.0, dtype=dtype, device=dev)
        eye = torch.eye(c, dtype=dtype, device=dev)
        Wo = torch.full((c, c), 1 / 1024, dtype=dtype, device=dev)  # 16 equal terms
        for pre in (False, True):
            out = sc.gated_ffn(x, torch.cat([eye, eye], 1).contiguous(), None, Wo, act="relu", return_pre=pre)
            out = (out[0] if pre else out).float()
            # two roundings at most, of h and of the result
            assert bool((out == ref).all()) if ref == float("inf") else bool(((out / ref - 1).abs() <= 2.1 * UB).all())
