"""Operators on the rows of packed items in fp64 numpy: group norm with an
activation, rotary positions, attention, and their gradients.

Written from the formulas, item by item; shares nothing with the library.
Offsets are host arrays [items + 1]; rows past the last belong to no item and
come out as zeros.
"""
from __future__ import annotations

import numpy as np

from .dense import act


def _items(offsets, n):
    offsets = [0, n] if offsets is None else [int(v) for v in offsets]
    return list(zip(offsets, offsets[1:]))


def group_norm(x, groups, w, b, eps, name, offsets=None):
    """(y, mean, rstd); w and b may be None."""
    x = np.asarray(x, np.float64)
    n, c = x.shape
    w = np.ones(c) if w is None else np.asarray(w, np.float64)
    b = np.zeros(c) if b is None else np.asarray(b, np.float64)
    y, stats = np.zeros_like(x), []
    for s, e in _items(offsets, n):
        t = x[s:e].reshape(e - s, groups, c // groups)
        m = t.mean((0, 2)) if e > s else np.zeros(groups)
        v = ((t - m[:, None]) ** 2).mean((0, 2)) if e > s else np.zeros(groups)
        r = 1 / np.sqrt(v + eps)
        y[s:e] = act(((t - m[:, None]) * r[:, None]).reshape(e - s, c) * w + b, name)[0]
        stats.append((m, r))
    return y, np.array([m for m, _ in stats]), np.array([r for _, r in stats])


def group_norm_backward(dy, x, mean, rstd, w, b, name, offsets=None):
    """(dx, dw, db)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    n, c = x.shape
    groups = mean.shape[1]
    w = np.ones(c) if w is None else np.asarray(w, np.float64)
    b = np.zeros(c) if b is None else np.asarray(b, np.float64)
    dx, dw, db = np.zeros_like(x), np.zeros(c), np.zeros(c)
    for i, (s, e) in enumerate(_items(offsets, n)):
        if e <= s:
            continue
        m, r = np.repeat(mean[i], c // groups), np.repeat(rstd[i], c // groups)
        xh = (x[s:e] - m) * r
        dz = dy[s:e] * act(xh * w + b, name)[1]
        dw += (dz * xh).sum(0)
        db += dz.sum(0)
        d = (dz * w).reshape(e - s, groups, -1)
        k = xh.reshape(e - s, groups, -1)
        g = d - d.mean((0, 2), keepdims=True) - k * (d * k).mean((0, 2), keepdims=True)
        dx[s:e] = g.reshape(e - s, c) * r
    return dx, dw, db


def rotary(x, positions, freqs, interleaved, inverse=False, amplitude=1.0):
    x = np.array(x, np.float64)
    at = np.asarray(positions, np.float64)
    at = at[:, None] if at.ndim == 1 else at
    p = at.shape[1] * len(freqs)
    t = (at[:, :, None] * np.asarray(freqs, np.float64)).reshape(x.shape[0], 1, p) * (-1 if inverse else 1)
    a, b = (slice(0, 2 * p, 2), slice(1, 2 * p, 2)) if interleaved else (slice(0, p), slice(p, 2 * p))
    u, v = x[:, :, a].copy(), x[:, :, b].copy()
    x[:, :, a] = amplitude * (u * np.cos(t) - v * np.sin(t))
    x[:, :, b] = amplitude * (v * np.cos(t) + u * np.sin(t))
    return x


def weights(q, k, scale, causal):
    """Softmax weights [Lq,Lk] and log sum exp [Lq] of one head of one item."""
    lq, lk = len(q), len(k)
    s = scale * (q @ k.T)
    if causal:
        s = np.where(np.arange(lk) <= np.arange(lq)[:, None] + lk - lq, s, -np.inf)
    top = s.max(1, initial=-np.inf)
    p = np.exp(s - np.where(np.isinf(top), 0.0, top)[:, None])
    total = p.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, top + np.log(total), -np.inf)
    return p / np.where(total > 0, total, 1.0)[:, None], lse


def _each(q, k, offsets, k_offsets, k_lengths):
    """(rows, keys, head, key head) of every item and head."""
    group = q.shape[1] // k.shape[1]
    keys = _items(offsets if k_offsets is None else k_offsets, k.shape[0])
    for i, (s, e) in enumerate(_items(offsets, q.shape[0])):
        ks, ke = keys[i]
        if k_lengths is not None:
            ke = min(ke, ks + max(0, int(k_lengths[i])))
        for h in range(q.shape[1]):
            yield slice(s, e), slice(ks, ke), h, h // group


def attention(q, k, v, scale, causal, offsets=None, k_offsets=None, k_lengths=None):
    """(out, lse)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    out, lse = np.zeros_like(q), np.full(q.shape[:2], -np.inf)
    for rows, keys, h, kh in _each(q, k, offsets, k_offsets, k_lengths):
        p, lse[rows, h] = weights(q[rows, h], k[keys, kh], scale, causal)
        out[rows, h] = p @ v[keys, kh]
    return out, lse


def attention_backward(do, q, k, v, out, scale, causal, offsets=None, k_offsets=None, k_lengths=None):
    """(dq, dk, dv), with delta from `out` as it was stored."""
    do, q, k, v, out = (np.asarray(t, np.float64) for t in (do, q, k, v, out))
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for rows, keys, h, kh in _each(q, k, offsets, k_offsets, k_lengths):
        p, _ = weights(q[rows, h], k[keys, kh], scale, causal)
        delta = (do[rows, h] * out[rows, h]).sum(1)
        ds = scale * p * (do[rows, h] @ v[keys, kh].T - delta[:, None])
        dq[rows, h] = ds @ k[keys, kh]
        dk[keys, kh] += ds.T @ q[rows, h]
        dv[keys, kh] += p.T @ do[rows, h]
    return dq, dk, dv
