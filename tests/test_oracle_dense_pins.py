"""The fp64 oracle of the dense layers against independent statements: torch's
modules on the CPU, and central differences of the forward for every gradient.

Differences: a central difference of step t has a truncation error of t^2 / 6
times a third derivative and a rounding error of 2^-52 |L| / t. With t = 1e-5,
losses of order 10 and third derivatives of order 10 both are near 1e-9; the
gradients are compared at 1e-6 (absolute and relative)."""
import numpy as np
import pytest
import torch

from oracle import dense as od

T = 1e-5


def _rng(seed):
    return np.random.default_rng(seed)


def _differences(loss, a):
    g = np.zeros_like(a)
    flat, out = a.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        v = flat[i]
        flat[i] = v + T
        up = loss()
        flat[i] = v - T
        down = loss()
        flat[i] = v
        out[i] = (up - down) / (2 * T)
    return g


def _close(got, ref):
    np.testing.assert_allclose(got, ref, rtol=1e-6, atol=1e-6)


def test_activations_equal_torch():
    z = np.linspace(-9, 9, 401)
    t = torch.from_numpy(z)
    F = torch.nn.functional
    for name, f in (("relu", F.relu), ("silu", F.silu), ("gelu", F.gelu),
                    ("gelu_tanh", lambda v: F.gelu(v, approximate="tanh")), ("none", lambda v: v)):
        np.testing.assert_allclose(od.act(z, name)[0], f(t).numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("name", od.ACTS)
def test_activation_slopes_equal_differences(name):
    z = np.array([-6.0, -2.3, -0.7, 0.2, 1.1, 4.0])
    ref = (od.act(z + T, name)[0] - od.act(z - T, name)[0]) / (2 * T)
    _close(od.act(z, name)[1], ref)


@pytest.mark.parametrize("n,c", [(1, 1), (3, 5), (4, 16)])
def test_layer_norm(n, c):
    r = _rng(n * 100 + c)
    x, w, b, dy = r.standard_normal((n, c)) + 0.5, r.standard_normal(c), r.standard_normal(c), r.standard_normal((n, c))
    y, m, rs = od.layer_norm(x, w, b, 1e-3)
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (c,), torch.from_numpy(w), torch.from_numpy(b), 1e-3)
    np.testing.assert_allclose(y, ref.numpy(), rtol=1e-10, atol=1e-10)
    dx, dw, db = od.layer_norm_backward(dy, x, m, rs, w)

    def loss():
        return (od.layer_norm(x, w, b, 1e-3)[0] * dy).sum()

    _close(dx, _differences(loss, x))
    _close(dw, _differences(loss, w))
    _close(db, _differences(loss, b))


@pytest.mark.parametrize("name", od.ACTS)
def test_linear(name):
    r = _rng(3)
    x, W, b = r.standard_normal((5, 4)), r.standard_normal((4, 6)), r.standard_normal(6)
    res, dy = r.standard_normal((5, 6)), r.standard_normal((5, 6))
    z = od.linear(x, W, b, name, res)[1]
    dx, dW, db, _ = od.linear_backward(dy, x, W, z, name)

    def loss():
        return (od.linear(x, W, b, name, res)[0] * dy).sum()

    for got, a in ((dx, x), (dW, W), (db, b), (dy, res)):
        _close(got, _differences(loss, a))


@pytest.mark.parametrize("name", od.ACTS)
def test_gated_ffn(name):
    r = _rng(4)
    x, Wi, bi = r.standard_normal((5, 4)), r.standard_normal((4, 6)), r.standard_normal(6)
    Wo, bo, res, dy = r.standard_normal((3, 2)), r.standard_normal(2), r.standard_normal((5, 2)), r.standard_normal((5, 2))
    z = od.gated_ffn(x, Wi, bi, Wo, bo, name, res)[1]
    dx, dWi, dbi, dWo, dbo, _, _ = od.gated_ffn_backward(dy, x, Wi, Wo, z, name)

    def loss():
        return (od.gated_ffn(x, Wi, bi, Wo, bo, name, res)[0] * dy).sum()

    for got, a in ((dx, x), (dWi, Wi), (dbi, bi), (dWo, Wo), (dbo, bo), (dy, res)):
        _close(got, _differences(loss, a))
