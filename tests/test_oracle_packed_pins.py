"""The fp64 oracle of the operators on packed items against independent
statements: torch's functions on the CPU, rotations as complex products, and
central differences of the forward for every gradient (steps and bounds as for
the dense layers: a difference is good to about 1e-9, compared at 1e-6)."""
import numpy as np
import pytest
import torch

from oracle import packed as op

T = 1e-5


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


def test_group_norm_equals_torch():
    r = np.random.default_rng(1)
    x, w, b = r.standard_normal((40, 12)), r.standard_normal(12), r.standard_normal(12)
    off = [0, 7, 7, 39]
    y, mean, _ = op.group_norm(x, 4, w, b, 1e-5, "silu", off)
    for s, e in ((0, 7), (7, 39)):
        t = torch.from_numpy(x[s:e].T[None])  # torch: [items, channels, positions]
        ref = torch.nn.functional.silu(
            torch.nn.functional.group_norm(t, 4, torch.from_numpy(w), torch.from_numpy(b), 1e-5))
        np.testing.assert_allclose(y[s:e], ref[0].numpy().T, rtol=1e-12, atol=1e-12)
    assert not y[39:].any() and not mean[1].any()


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_group_norm_gradients(name):
    r = np.random.default_rng(2)
    x, w, b, g = r.standard_normal((9, 6)), r.standard_normal(6), r.standard_normal(6), r.standard_normal((9, 6))
    off = [0, 3, 3, 8]
    _, mean, rstd = op.group_norm(x, 3, w, b, 1e-3, name, off)
    dx, dw, db = op.group_norm_backward(g, x, mean, rstd, w, b, name, off)

    def loss():
        return (g * op.group_norm(x, 3, w, b, 1e-3, name, off)[0]).sum()

    _close(dx, _differences(loss, x))
    _close(dw, _differences(loss, w))
    _close(db, _differences(loss, b))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_complex_product(interleaved):
    r = np.random.default_rng(3)
    x, at, f = r.standard_normal((5, 2, 14)), r.integers(-50, 50, (5, 3)), np.array([1.0, 0.1])
    y = op.rotary(x, at, f, interleaved)
    angle = np.concatenate([at[:, a:a + 1] * f for a in range(3)], 1)  # axis by axis
    z = x[:, :, 0:12:2] + 1j * x[:, :, 1:12:2] if interleaved else x[:, :, :6] + 1j * x[:, :, 6:12]
    z = z * np.exp(1j * angle)[:, None]
    np.testing.assert_allclose(y[:, :, 0:12:2] if interleaved else y[:, :, :6], z.real, atol=1e-12)
    np.testing.assert_allclose(y[:, :, 1:12:2] if interleaved else y[:, :, 6:12], z.imag, atol=1e-12)
    assert np.array_equal(y[:, :, 12:], x[:, :, 12:])
    np.testing.assert_allclose(op.rotary(y, at, f, interleaved, inverse=True), x, atol=1e-12)
    g = r.standard_normal(x.shape)
    _close(op.rotary(g, at, f, interleaved, inverse=True),
           _differences(lambda: (g * op.rotary(x, at, f, interleaved)).sum(), x))


@pytest.mark.parametrize("causal", [False, True])
def test_attention_equals_torch(causal):
    r = np.random.default_rng(4)
    q, k, v = r.standard_normal((11, 4, 8)), r.standard_normal((11, 2, 8)), r.standard_normal((11, 2, 8))
    off = [0, 5, 5, 10]
    out, lse = op.attention(q, k, v, 0.3, causal, off)
    for s, e in ((0, 5), (5, 10)):
        t = [torch.from_numpy(a[s:e]).transpose(0, 1) for a in (q, k.repeat(2, 1), v.repeat(2, 1))]
        ref = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=causal, scale=0.3)
        np.testing.assert_allclose(out[s:e], ref.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)
    assert not out[10:].any() and np.isneginf(lse[10:]).all()


def test_attention_masks_from_the_end_and_leaves_rows_empty():
    r = np.random.default_rng(5)
    q, k, v = r.standard_normal((4, 1, 8)), r.standard_normal((2, 1, 8)), r.standard_normal((2, 1, 8))
    out, lse = op.attention(q, k, v, 1.0, True, [0, 4], [0, 2])
    assert not out[:2].any() and np.isneginf(lse[:2]).all()  # two keys for four queries
    np.testing.assert_allclose(out[2], v[0])
    one, _ = op.attention(q, k, v, 1.0, False, [0, 4], [0, 2], [1])
    np.testing.assert_allclose(one, np.broadcast_to(v[0], one.shape))


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradients(causal):
    r = np.random.default_rng(6)
    q, k, v = r.standard_normal((6, 2, 4)), r.standard_normal((5, 1, 4)), r.standard_normal((5, 1, 4))
    off, koff, lengths = [0, 2, 5], [0, 3, 5], [2, 2]
    g = r.standard_normal(q.shape)

    def loss():
        return (g * op.attention(q, k, v, 0.7, causal, off, koff, lengths)[0]).sum()

    out, _ = op.attention(q, k, v, 0.7, causal, off, koff, lengths)
    grads = op.attention_backward(g, q, k, v, out, 0.7, causal, off, koff, lengths)
    for got, a in zip(grads, (q, k, v)):
        _close(got, _differences(loss, a))
