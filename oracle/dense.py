"""Dense layers of a sparse block in fp64 numpy: layer norm, linear with
activation and residual, the gated feed-forward block, and their gradients.

Written from the formulas; shares nothing with the library.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erf, expit

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(z, name):
    """Activation and its derivative."""
    z = np.asarray(z, np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, z, 0.0), (z > 0).astype(np.float64)
    if name == "silu":
        p = expit(z)
        return z * p, p + z * p * expit(-z)
    if name == "gelu":
        c = 0.5 * (1.0 + erf(z / np.sqrt(2.0)))
        return z * c, c + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        k = np.sqrt(2.0 / np.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    raise ValueError(name)


def layer_norm(x, w, b, eps):
    """(y, mean, rstd); w and b may be None."""
    x = np.asarray(x, np.float64)
    m = x.mean(1)
    r = 1.0 / np.sqrt(((x - m[:, None]) ** 2).mean(1) + eps)
    y = (x - m[:, None]) * r[:, None]
    y = y * (1.0 if w is None else np.asarray(w, np.float64))
    return y + (0.0 if b is None else np.asarray(b, np.float64)), m, r


def layer_norm_backward(dy, x, mean, rstd, w):
    """(dx, dw, db)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * r
    d = dy * (1.0 if w is None else np.asarray(w, np.float64))
    dx = r * (d - d.mean(1, keepdims=True) - xh * (d * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def linear(x, W, b, name, residual):
    """(out, z)."""
    z = np.asarray(x, np.float64) @ np.asarray(W, np.float64)
    if b is not None:
        z = z + np.asarray(b, np.float64)
    out = act(z, name)[0]
    return out + (0.0 if residual is None else np.asarray(residual, np.float64)), z


def linear_backward(dy, x, W, z, name):
    """(dx, dW, db, dz)."""
    dz = np.asarray(dy, np.float64)
    if name != "none":
        dz = dz * act(z, name)[1]
    return dz @ np.asarray(W, np.float64).T, np.asarray(x, np.float64).T @ dz, dz.sum(0), dz


def gated_ffn(x, W_in, b_in, W_out, b_out, name, residual):
    """(out, [g | u], h)."""
    z = np.asarray(x, np.float64) @ np.asarray(W_in, np.float64)
    if b_in is not None:
        z = z + np.asarray(b_in, np.float64)
    F = z.shape[1] // 2
    h = act(z[:, :F], name)[0] * z[:, F:]
    out = h @ np.asarray(W_out, np.float64)
    if b_out is not None:
        out = out + np.asarray(b_out, np.float64)
    return out + (0.0 if residual is None else np.asarray(residual, np.float64)), z, h


def gated_ffn_backward(dy, x, W_in, W_out, z, name):
    """(dx, dW_in, db_in, dW_out, db_out, dz, h)."""
    dy, x, z = (np.asarray(a, np.float64) for a in (dy, x, z))
    W_in, W_out = np.asarray(W_in, np.float64), np.asarray(W_out, np.float64)
    F = z.shape[1] // 2
    g, u = z[:, :F], z[:, F:]
    a, d = act(g, name)
    dh = dy @ W_out.T
    dz = np.concatenate([dh * u * d, dh * a], 1)
    h = a * u
    return dz @ W_in.T, x.T @ dz, dz.sum(0), h.T @ dy, dy.sum(0), dz, h
