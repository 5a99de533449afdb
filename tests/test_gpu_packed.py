"""The operators on packed items on the GPU (group norm with an activation, rotary
positions, attention, forward and backward) against the fp64 oracle, on the very
inputs the GPU reads.

Tolerances, per element, from the roundings that are made (u the unit roundoff of
the stored type: 2^-11 fp16, 2^-8 bf16, 2^-24 fp32; v = 2^-24):
- one rounding of a stored value: u |ref| (and 2^-24 for fp16 subnormals);
- a weight or score gradient rounded to 16 bits between two products carries u
  times itself into the next one; the fp16 ones below their smallest normal
  number 2^-25 of the scale they are held at;
- an fp32 sum of K products: at most (K + 4) v sum |a| |b|;
- a score's error e is a relative error e of its weight and of the row's sum;
- exp2, log2, reciprocal: a few v, and v times the size of exp2's argument;
- activations as for the dense layers: 32 v (1 + |z|) for value and slope, and a
  slope of at most 1.2 passes on the error of z;
- statistics joined from parts in at most J steps: J v times the values joined.
Every bound is the sum of such terms; none is fitted.
"""
import numpy as np
import pytest
import torch

from oracle import packed as op
from oracle.dense import act as act_ref

gpu = pytest.mark.gpu
V = 2.0 ** -24
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: V}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 1e-30, torch.float32: 1e-30}
TYPES = [torch.float16, torch.bfloat16, torch.float32]
IDS = ["fp16", "bf16", "fp32"]


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
    return t.detach().cpu().double().numpy()


def _check(got, ref, tol, what):
    got = _np(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    with np.errstate(invalid="ignore"):  # equal infinities
        bad = ~((got == ref) | (np.abs(got - ref) <= tol))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} x the bound")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(shape, dtype, dev, seed, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=_gen(seed)) * scale + shift).to(dtype).to(dev)


def _offsets(lengths, dev):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32).to(dev)


# ---------------------------------------------------------------------------
# item offsets
# ---------------------------------------------------------------------------


@gpu
@pytest.mark.parametrize("lengths", [[5], [0, 3], [3, 0, 0, 4], [300, 1, 700, 0], [0], [0, 0], [1] * 500, [70000, 5]])
def test_item_offsets(dev, lengths):
    sc = _sc()
    b = torch.arange(len(lengths)).repeat_interleave(torch.tensor(lengths))
    coords = torch.stack([b, b * 0 + 3, b * 0 - 1, b * 0 + 70000], 1).to(torch.int32).to(dev)
    got = sc.item_offsets(coords, len(lengths))
    assert got.dtype == torch.int32 and torch.equal(got.cpu(), _offsets(lengths, "cpu"))


@gpu
def test_item_offsets_refuses_what_is_not_sorted(dev):
    sc = _sc()
    coords = torch.zeros((600, 4), dtype=torch.int32, device=dev)
    coords[300:, 0] = 1
    assert sc.item_offsets(coords).tolist() == [0, 300, 600]
    bad = coords.clone()
    bad[400, 0] = 0
    with pytest.raises(sc.SubmconvError, match="order"):
        sc.item_offsets(bad, 2)
    for v in (2, -1, 2 ** 31 - 1, -2 ** 31):
        bad = coords.clone()
        bad[599, 0] = v
        with pytest.raises(sc.SubmconvError, match="outside"):
            sc.item_offsets(bad, 2)


@gpu
@pytest.mark.parametrize("row", [0, 298, 299, 300])
@pytest.mark.parametrize("value", [2, 65535, 2 ** 31 - 1, -2 ** 31])
def test_item_offsets_refuses_an_index_anywhere(dev, row, value):
    sc = _sc()
    coords = torch.zeros((600, 4), dtype=torch.int32, device=dev)
    coords[300:, 0] = 1
    coords[row, 0] = value
    with pytest.raises(sc.SubmconvError, match="outside"):
        sc.item_offsets(coords, 2)


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

# rows per item (and rows behind the last), channels, groups, columns of padding
NORMS = [([1], 0, 8, 1, 0), ([7], 0, 32, 32, 0), ([64, 0], 3, 256, 32, 0), ([20, 300, 1], 5, 60, 12, 3),
         ([0, 0], 4, 16, 2, 0), ([700, 321], 0, 128, 32, 8), ([1023], 1, 64, 1, 0), ([5] * 90, 0, 24, 8, 1),
         ([3000], 0, 128, 32, 0), ([1500, 0, 2500, 1], 77, 60, 12, 3), ([2100], 9, 33, 3, 1), ([1100, 5], 0, 515, 5, 0),
         ([1300], 0, 2056, 8, 0), ([900, 200], 0, 4100, 1, 2), ([1025], 0, 8192, 64, 0), ([700, 700], 3, 8192, 8192, 0),
         ([0, 1200, 0], 100, 20, 20, 0), ([3] * 400, 1, 8, 2, 0), ([0], 0, 16, 4, 0),
         ([40] * 100 + [0, 1, 5000], 3, 96, 8, 0), ([2] * 3000, 5, 40, 5, 0),
         ([100] * 127, 0, 40, 5, 0), ([60] * 128, 2, 64, 8, 0), ([9000] + [1] * 126, 0, 16, 2, 0), ([20000], 5, 33, 11, 0),
         ([0, 12000, 30], 0, 320, 32, 0)]


def _joins(lengths, c, groups):
    """Steps in which a group's sums come together (blocks of 4 rows, threads, channels, chunks), from above."""
    return max(list(lengths) + [1]) / 4 + 300 + c // groups


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", range(len(NORMS)))
def test_group_norm(dev, case, dtype):
    sc = _sc()
    lengths, behind, c, groups, pad = NORMS[case]
    act = ["silu", "none", "gelu", "relu", "gelu_tanh"][case % 5]
    n, eps = sum(lengths) + behind, 1e-5
    wide = torch.full((n, c + 2 * pad), float("nan"), dtype=dtype)
    wide[:, pad:pad + c] = (torch.randn((n, c), generator=_gen(case)) * 1.3 + 0.7).to(dtype)
    if behind:
        wide[n - behind:] = float("nan")  # rows of no item are not read
    x = wide.to(dev)[:, pad:pad + c]
    affine = case % 4 != 2
    w = _randn((c,), torch.float32, dev, 1, 0.3, 1.0) if affine else None
    b = _randn((c,), torch.float32, dev, 2, 0.3) if affine else None
    off = _offsets(lengths, dev) if len(lengths) > 1 or behind else None
    offn = None if off is None else off.tolist()
    y, mean, rstd = sc.group_norm(x, groups, w, b, eps, act, off, return_stats=True)
    assert torch.equal(y, sc.group_norm(x, groups, w, b, eps, act, off))  # and repeats bit for bit
    xn = np.where(np.isnan(_np(x)), 0.0, _np(x))
    ry, rm, rr = op.group_norm(xn, groups, w if w is None else _np(w), b if b is None else _np(b), eps, act, offn)
    wn, bn = (np.ones(c), np.zeros(c)) if w is None else (_np(w), _np(b))
    e = _joins(lengths, c, groups) * V
    top = np.array([[np.abs(xn[s:t].reshape(t - s, groups, c // groups)).max((0, 2), initial=0)] for s, t in op._items(offn, n)])
    em = e * top[:, 0]  # of the mean
    sd = np.sqrt(np.maximum(1 / rr ** 2 - eps, 0))
    er = rr * (2 * e + (2 * em * sd + em * em) * rr ** 2 + 4 * V)
    _check(mean, rm, em + V * np.abs(rm), "mean")
    _check(rstd, rr, er, "rstd")
    tol = np.full((n, c), 0.0)
    for i, (s, t) in enumerate(op._items(offn, n)):
        per = [np.repeat(a[i], c // groups) for a in (rm, rr, em, er)]
        a = np.abs(xn[s:t] - per[0])
        z = a * per[1] * np.abs(wn) + np.abs(bn)
        ez = np.abs(wn) * (a * per[3] + per[1] * (per[2] + 2 * V * (np.abs(xn[s:t]) + np.abs(per[0])))) + 4 * V * z
        tol[s:t] = 1.2 * ez + 32 * V * (1 + z) + U[dtype] * np.abs(ry[s:t]) + TINY[dtype]
    _check(y, ry, tol, "y")

    # gradients, for the statistics that the forward wrote
    dy = torch.randn((n, c), generator=_gen(100 + case)).to(dtype).to(dev)
    gx, gw, gb = sc.group_norm_backward(dy, x, mean, rstd, w, b, act, off)
    dyn, mn, rn = _np(dy), _np(mean), _np(rstd)
    rx, rw, rb = op.group_norm_backward(dyn, xn, mn, rn, wn, bn, act, offn)
    tw, tb, tx = np.zeros(c), np.zeros(c), np.zeros((n, c))
    for i, (s, t) in enumerate(op._items(offn, n)):
        if t <= s:
            continue
        m, r = np.repeat(mn[i], c // groups), np.repeat(rn[i], c // groups)
        xh = (xn[s:t] - m) * r
        exh = 4 * V * (np.abs(xn[s:t]) + np.abs(m)) * r
        z = xh * wn + bn
        slope = act_ref(z, act)[1]
        ez = exh * np.abs(wn) + 2 * V * (np.abs(xh * wn) + np.abs(bn))
        # of the slope: it changes by at most 1.2 per unit of z; relu's jumps, where z is near 0
        es = 1.2 * ez + 32 * V * (1 + np.abs(z)) if act != "relu" else np.where(np.abs(z) <= ez, 1.0, 0.0)
        if act == "none":
            es = 0 * ez
        edz = np.abs(dyn[s:t]) * (es + 2 * V)
        dz = np.abs(dyn[s:t] * slope)
        k = (t - s) / 4 + 300
        tb += edz.sum(0) + k * V * dz.sum(0)
        tw += (edz * np.abs(xh) + dz * exh).sum(0) + k * V * (dz * np.abs(xh)).sum(0)
        d, ed = dz * np.abs(wn), edz * np.abs(wn) + V * dz * np.abs(wn)
        shape = (t - s, groups, c // groups)

        def mean_of(a):
            return np.repeat(a.reshape(shape).mean((0, 2)), c // groups)

        kk = k + c // groups
        e1 = mean_of(ed) + kk * V * mean_of(d)
        s2 = mean_of(d * np.abs(xh))
        e2 = mean_of(ed * np.abs(xh) + d * exh) + kk * V * s2
        tx[s:t] = r * (ed + e1 + np.abs(xh) * e2 + exh * s2 + 8 * V * (d + mean_of(d) + np.abs(xh) * s2))
    _check(gx, rx, tx + U[dtype] * np.abs(rx) + TINY[dtype], "grad_x")
    _check(gw, rw, tw + 1e-30, "grad_weight")
    _check(gb, rb, tb + 1e-30, "grad_bias")
    only = sc.group_norm_backward(dy, x, mean, rstd, w, b, act, off, needs=(False, True, False))
    assert only[0] is None and only[2] is None and torch.equal(only[1], gw)
    only = sc.group_norm_backward(dy, x, mean, rstd, w, b, act, off, needs=(True, False, False))
    assert only[1] is None and only[2] is None and torch.equal(only[0], gx)


@gpu
@pytest.mark.parametrize("n", [500, 5000])
def test_group_norm_far_from_zero_and_constant_items(dev, n):
    """A mean of 1000 deviations keeps its variance; a constant item has variance 0
    and y = act(bias)."""
    sc = _sc()
    x = torch.randn((2 * n, 32), generator=_gen(5)) + 1000.0
    x[n:] = 3.0
    b = torch.linspace(-1, 1, 32)
    y, _, rstd = sc.group_norm(x.to(dev), 4, None, b.to(dev), act="relu", offsets=_offsets([n, n], dev),
                               return_stats=True)
    ry, _, rr = op.group_norm(x.numpy(), 4, None, b.numpy(), 1e-5, "relu", [0, n, 2 * n])
    # the mean: (n / 4 + 308) v 1000, and as much relative to the deviation 1
    e = (n / 4 + 308) * V * 1000
    _check(y, ry, 2 * e * (1 + np.abs(ry)), "y")
    assert torch.equal(y[n:].cpu(), b.clamp(min=0).expand(n, 32))


@gpu
def test_group_norm_gradient_against_differences(dev):
    """fp32, along one direction: (f(x + t d) - f(x - t d)) / 2t. With t = 2^-6 its
    truncation is t^2 / 6 times a third derivative of order 1 per unit direction,
    1e-4 relative to the sum of the terms' sizes; fp32 values of size 1 leave
    2 v / t = 8e-6 of it. Bound: 1e-3 of the norms' product."""
    sc = _sc()
    n, c, off = 1500, 24, _offsets([600, 900], dev)
    x, d, g = (_randn((n, c), torch.float32, dev, s) for s in (1, 2, 3))
    w, b = _randn((c,), torch.float32, dev, 4, 0.2, 1.0), _randn((c,), torch.float32, dev, 5, 0.2)

    def f(t):
        return (sc.group_norm(x + t * d, 4, w, b, act="silu", offsets=off).double() * g.double()).sum().item()

    _, mean, rstd = sc.group_norm(x, 4, w, b, act="silu", offsets=off, return_stats=True)
    gx, _, _ = sc.group_norm_backward(g, x, mean, rstd, w, b, "silu", off)
    t = 2.0 ** -6
    slope = (gx.double() * d.double()).sum().item()
    assert abs((f(t) - f(-t)) / (2 * t) - slope) <= 1e-3 * (gx.norm() * d.norm()).item()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

# rows, heads, columns, axes, rotated columns, positions up to
TURNS = [(1, 1, 2, 1, 2, 5), (1, 16, 64, 1, 64, 131072), (7, 3, 80, 1, 48, 2 ** 31 - 1), (300, 5, 64, 3, 60, 512),
         (33, 2, 96, 3, 96, 100), (65, 1, 20, 4, 16, 9), (5, 7, 33, 1, 14, 70), (20000, 2, 64, 1, 64, 20000),
         (0, 4, 32, 1, 32, 4), (3, 300, 128, 2, 100, 1000)]


@gpu
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("case", range(len(TURNS)))
def test_rotary(dev, case, dtype, interleaved):
    sc = _sc()
    n, h, d, axes, part, reach = TURNS[case]
    wide = _randn((n, h + 3, d + 1), dtype, dev, case)
    x = wide[:, 1:h + 1, :d]
    at = torch.randint(-reach, reach, (n, axes + 1), generator=_gen(case), dtype=torch.int32).to(dev)[:, 1:]
    f = sc.rotary_frequencies(part, axes, device=dev)
    at1 = at[:, 0] if axes == 1 else at
    y = sc.rotary(x, at1, f, interleaved, amplitude=1.25)
    ref = op.rotary(_np(x), _np(at), _np(f), interleaved, amplitude=1.25)
    # angle: two fp64 roundings of up to 2^31 / 2 pi turns (2^-24 turns), fp32 of the part of a turn
    # (2^-25 turns), so 2 pi 2^-23 in all; sine and cosine 4 v; three roundings of the sum
    size = np.abs(_np(x))
    pairs = part // 2
    a, b = (slice(0, part, 2), slice(1, part, 2)) if interleaved else (slice(0, pairs), slice(pairs, part))
    both = size[:, :, a] + size[:, :, b]
    tol = np.zeros_like(ref)
    tol[:, :, a] = tol[:, :, b] = 1.25 * both * (2 * np.pi * 2 * V + 12 * V)
    _check(y, ref, tol + np.where(tol > 0, U[dtype] * np.abs(ref) + TINY[dtype], 0), "y")
    back = sc.rotary(x, at1, f, interleaved, inverse=True)
    _check(back, op.rotary(_np(x), _np(at), _np(f), interleaved, inverse=True),
           tol + np.where(tol > 0, U[dtype] * np.abs(ref) + U[dtype] * both.max(initial=1) + TINY[dtype], 0), "inverse")
    # in place: the same values, and nothing beside them is touched
    before = wide.clone()
    got = sc.rotary(x, at1, f, interleaved, amplitude=1.25, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(x, y)
    before[:, 1:h + 1, :d] = y
    assert torch.equal(wide, before)


@gpu
def test_rotary_frequencies_and_function(dev):
    sc = _sc()
    f = sc.rotary_frequencies(64)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    np.testing.assert_allclose(sc.rotary_frequencies(64, scaling="linear", factor=4).numpy(), f.numpy() / 4)
    g = sc.rotary_frequencies(64, scaling="base", factor=4).numpy()
    assert g[0] == 1.0 and abs(g[-1] / (f[-1].item() / 4) - 1) < 1e-12  # the slowest is divided by the factor
    p = sc.rotary_frequencies(64, scaling="parts", factor=4).numpy()
    turns = 4096 * f.numpy() / (2 * np.pi)
    np.testing.assert_allclose(p[turns > 32], f.numpy()[turns > 32])
    np.testing.assert_allclose(p[turns < 1], f.numpy()[turns < 1] / 4)
    assert ((p >= f.numpy() / 4) & (p <= f.numpy())).all()
    x = _randn((9, 2, 64), torch.float32, dev, 3).requires_grad_()
    at = torch.arange(9, device=dev, dtype=torch.int32)
    y = sc.RotaryFunction.apply(x, at, f.to(dev), True, 1.0)
    grad = _randn((9, 2, 64), torch.float32, dev, 4)
    y.backward(grad)
    # a rotation: the gradient of <y, grad> along x is <grad, y>
    assert abs((x.grad * x).sum() - (grad * y).sum()).item() < 1e-3


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

# rows per item, keys per item (None: the same rows), rows behind, heads, key heads, columns, causal
ATTN = [
    ([1], None, 0, 1, 1, 8, False), ([5], None, 0, 2, 1, 32, True), ([64], None, 0, 2, 2, 64, True),
    ([65, 63], None, 1, 3, 3, 64, False), ([130], None, 0, 4, 2, 128, True), ([100, 0, 1, 77], None, 9, 4, 1, 40, True),
    ([129, 200], None, 0, 2, 2, 96, False), ([33, 300], None, 3, 6, 2, 72, True), ([257], None, 0, 9, 9, 16, False),
    ([300, 17], None, 0, 16, 8, 128, False), ([31, 1], None, 0, 8, 8, 24, True),
    ([50, 20, 0], [7, 90, 4], 2, 2, 1, 64, True),      # more queries than keys: rows that see nothing
    ([40, 3], [0, 65], 0, 2, 2, 32, False),            # an item without keys
    ([10, 200], [500, 0], 0, 4, 4, 112, True), ([300, 100], [77, 77], 0, 5, 5, 72, False),
    ([1, 1, 1], [700, 1, 64], 0, 16, 2, 64, True),     # one new token each over its cache
    ([1] * 5, [300, 0, 129, 65, 1000], 0, 8, 1, 128, True), ([2, 3], [2000, 1500], 0, 4, 4, 96, True),
    ([4], [9000], 0, 2, 2, 64, False),                 # the keys are split
    ([1500], [70], 0, 1, 1, 64, False),                # the queries are split in the gradient of the keys
    ([600], None, 0, 1, 1, 128, True),
]


def _attn_case(case, dtype, dev, scale=1.3):
    lengths, keys, behind, h, hk, d, causal = ATTN[case]
    n = sum(lengths) + behind
    off = _offsets(lengths, dev) if len(lengths) > 1 or behind else None
    if keys is None:
        nk, koff = n, None
        q, k, v = _randn((n, h + 2 * hk, d), dtype, dev, case, scale).split([h, hk, hk], 1)
    else:
        nk, koff = sum(keys) + 3, _offsets(keys, dev)
        off = _offsets(lengths, dev)
        q = _randn((n, h, d), dtype, dev, case, scale)
        k, v = _randn((nk, 2 * hk, d), dtype, dev, case + 1000, scale).split([hk, hk], 1)
        k[nk - 3:], v[nk - 3:] = float("nan"), float("inf")  # rows of no item are not read
    if behind:
        q[n - behind:] = float("nan")
        if keys is None:
            k[n - behind:], v[n - behind:] = float("nan"), float("nan")
    return q, k, v, off, koff, causal


def _clean(t):
    return np.where(np.isfinite(_np(t)), _np(t), 0.0)


def _bounds(q, k, v, out, do, scale, causal, off, koff, klen, dtype):
    """Bounds of out, lse and the three gradients from the terms in the head of
    this file; gradients for `out` and `lse` as the forward wrote them."""
    u, half = U[dtype], dtype == torch.float16
    d = q.shape[2]
    to, tl = np.zeros_like(q), np.zeros(q.shape[:2])
    tq, tk, tv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for rows, keys, h, kh in op._each(q, k, off, koff, klen):
        qq, kk, vv = q[rows, h], k[keys, kh], v[keys, kh]
        p, lse = op.weights(qq, kk, scale, causal)
        nk = p.shape[1]
        if p.size == 0:
            continue
        on = p > 0
        s = np.abs(scale * (qq @ kk.T)) * on
        es = ((d + 4) * V * scale * (np.abs(qq) @ np.abs(kk).T) + 4 * V * s) * on
        # of a weight, relative: its score's, the row's largest score's, exp2's argument
        size = s.max(1, keepdims=True)
        ep = es + 8 * V + 4 * V * (s + size)
        esum = ep.max(1, keepdims=True) + (nk + 8) * V
        av = np.abs(vv)
        to[rows, h] = (p * (u + ep + esum + (nk + 32) * V)) @ av + (2.0 ** -25 * on @ av if half else 0)
        tl[rows, h] = esum[:, 0] + 8 * V * (1 + size[:, 0] + np.log(nk + 1))
        if do is None:
            continue
        dd, oo = do[rows, h], out[rows, h]
        eg = es + tl[rows, h][:, None] + 8 * V + 4 * V * (s + np.where(np.isinf(lse), 0, np.abs(lse))[:, None])
        dp = dd @ vv.T
        delta = (dd * oo).sum(1, keepdims=True)
        edp = (d + 4) * V * (np.abs(dd) @ av.T + (np.abs(dd) * np.abs(oo)).sum(1, keepdims=True)) + 2 * V * np.abs(dp)
        ds = np.abs(p * (dp - delta))
        # rounding of ds; in fp16 what is below the normal numbers: 2^-25 at a scale where the
        # column's largest so far is at least 2^7
        eds = ds * (u + eg + 4 * V) + p * edp
        low = 2.0 ** -32 if half else 0.0
        n_q = p.shape[0]
        tq[rows, h] = scale * ((eds + (nk + 8) * V * ds + low * ds.max(1, keepdims=True)) @ np.abs(kk))
        tk[keys, kh] += scale * ((eds + (n_q + 8) * V * ds + low * ds.max(0, keepdims=True)).T @ np.abs(qq))
        tv[keys, kh] += (p * (u + eg + (n_q + 8) * V) + (2.0 ** -37 if half else 0)).T @ np.abs(dd)
    return to, tl, tq, tk, tv


@gpu
@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(dev, case, dtype):
    sc = _sc()
    q, k, v, off, koff, causal = _attn_case(case, dtype, dev)
    scale = None if case % 2 else 0.21
    out, lse = sc.attention(q, k, v, off, koff, causal=causal, scale=scale, return_lse=True)
    assert torch.equal(out, sc.attention(q, k, v, off, koff, causal=causal, scale=scale))  # bit for bit
    scale = np.float32(q.shape[2] ** -0.5 if scale is None else scale).astype(np.float64)
    offn, koffn = (None if t is None else t.tolist() for t in (off, koff))
    qn, kn, vn = _clean(q), _clean(k), _clean(v)
    ro, rl = op.attention(qn, kn, vn, scale, causal, offn, koffn)
    do = _randn(tuple(q.shape), dtype, dev, 77 + case)
    don = _np(do)
    to, tl, tq, tk, tv = _bounds(qn, kn, vn, _np(out), don, scale, causal, offn, koffn, None, dtype)
    _check(out, ro, to + U[dtype] * np.abs(ro) + TINY[dtype], "out")
    _check(lse, rl, tl, "lse")
    grads = sc.attention_backward(do, q, k, v, out, lse, off, koff, causal=causal, scale=float(scale))
    for a, b in zip(grads, sc.attention_backward(do, q, k, v, out, lse, off, koff, causal=causal, scale=float(scale))):
        assert torch.equal(a, b)
    refs = op.attention_backward(don, qn, kn, vn, _np(out), scale, causal, offn, koffn)
    for got, ref, tol, what in zip(grads, refs, (tq, tk, tv), ("grad_q", "grad_k", "grad_v")):
        _check(got, ref, tol + U[dtype] * np.abs(ref) + TINY[dtype], what)
    for need in range(3):
        needs = [i == need for i in range(3)]
        some = sc.attention_backward(do, q, k, v, out, lse, off, koff, causal=causal, scale=float(scale), needs=needs)
        assert [t is not None for t in some] == needs and torch.equal(some[need], grads[need])


@gpu
@pytest.mark.parametrize("causal", [False, True])
def test_attention_heads_of_rows(dev, causal):
    """Tensors stored head by head, and a single row or head with any stride, give
    what rows of heads give."""
    sc = _sc()
    n, h, hk, d = 150, 4, 2, 64
    q, k, v, g = (_randn((n, a, d), torch.float16, dev, s) for a, s in ((h, 1), (hk, 2), (hk, 3), (h, 4)))
    out, lse = sc.attention(q, k, v, causal=causal, return_lse=True)
    grads = sc.attention_backward(g, q, k, v, out, lse, causal=causal)
    tq, tk, tv, tg = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, g))
    assert tq.stride() == (d, n * d, 1)
    assert torch.equal(sc.attention(tq, tk, tv, causal=causal), out)
    for a, b in zip(sc.attention_backward(tg, tq, tk, tv, out, lse, causal=causal), grads):
        assert torch.equal(a, b)
    at, f = torch.arange(n, dtype=torch.int32, device=dev), sc.rotary_frequencies(32, device=dev)
    y = torch.empty_like(tq)
    assert torch.equal(sc.rotary(tq, at, f, out=y), sc.rotary(q, at, f)) and y.stride() == tq.stride()
    one = sc.attention(q[:1, :2], k[:1, :1], v[:1, :1])
    odd = [torch.empty_strided(t.shape, (7, t.shape[2], 1), dtype=t.dtype, device=dev).copy_(t)
           for t in (q[:1, :2], k[:1, :1], v[:1, :1])]
    assert torch.equal(sc.attention(*odd), one)
    with pytest.raises(ValueError, match="overlap"):
        sc.attention(q, k[:, :1].expand(n, 2, d), v)


@gpu
def test_attention_with_nothing_on_a_side(dev):
    sc = _sc()
    h, hk, d = 4, 2, 32
    some, none = torch.tensor([0, 3, 5], dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    q, k = _randn((5, h, d), torch.float16, dev, 1), _randn((5, hk, d), torch.float16, dev, 2)
    out, lse = sc.attention(q, k[:0], k[:0], some, none, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    dq, dk, dv = sc.attention_backward(q, q, k[:0], k[:0], out, lse, some, none)
    assert not dq.any() and dk.shape == dv.shape == (0, hk, d)
    out, lse = sc.attention(q[:0], k, k, none, some, return_lse=True)
    assert out.shape == (0, h, d) and lse.shape == (0, h)
    dq, dk, dv = sc.attention_backward(q[:0], q[:0], k, k, out, lse, none, some)
    assert dq.shape == (0, h, d) and not dk.any() and not dv.any()
    assert sc.attention(q[:0], k[:0], k[:0]).shape == (0, h, d)


@gpu
@pytest.mark.parametrize("items", [64, 65, 700])
def test_attention_of_many_items(dev, items):
    """Lengths of 0 to 40 in any order, under the causal mask: up to 64 items the
    tiles go by their walks, past that item by item."""
    sc = _sc()
    g = _gen(items)
    lengths = torch.randint(0, 41, (items,), generator=g).tolist()
    lengths[items // 2] = 600
    n, h, hk, d = sum(lengths) + 7, 4, 1, 32
    q, k, v = (_randn((n, a, d), torch.float16, dev, s) for a, s in ((h, 1), (hk, 2), (hk, 3)))
    off = _offsets(lengths, dev)
    out, lse = sc.attention(q, k, v, off, causal=True, return_lse=True)
    args = (d ** -0.5, True, off.tolist(), None)
    ro, rl = op.attention(_np(q), _np(k), _np(v), *args)
    do = _randn((n, h, d), torch.float16, dev, 4)
    to, tl, tq, tk, tv = _bounds(_np(q), _np(k), _np(v), _np(out), _np(do), *args, None, torch.float16)
    _check(out, ro, to + 2.0 ** -11 * np.abs(ro) + 2.0 ** -24, "out")
    _check(lse, rl, tl, "lse")
    grads = sc.attention_backward(do, q, k, v, out, lse, off, causal=True)
    refs = op.attention_backward(_np(do), _np(q), _np(k), _np(v), _np(out), *args)
    for got, ref, tol, what in zip(grads, refs, (tq, tk, tv), ("grad_q", "grad_k", "grad_v")):
        _check(got, ref, tol + 2.0 ** -11 * np.abs(ref) + 2.0 ** -24, what)


@gpu
def test_attention_of_offsets_that_descend_stays_in_bounds(dev):
    """What they mean is undefined; rows beside the tensors stay as they are, and
    the kernels end. (Kernels cut offsets to 0 .. n, whatever they hold.)"""
    sc = _sc()
    n, h, d = 300, 2, 32
    wide = _randn((n + 20, h, d), torch.float16, dev, 1)
    q = wide[10:n + 10]
    before = wide.clone()
    for bad in ([0, 200, 100, 300], [5, -7, 2 ** 31 - 1, 40], [0, 400, 500, 600]):
        off = torch.tensor(bad, dtype=torch.int32, device=dev)
        for causal in (False, True):
            out, lse = sc.attention(q, q, q, off, causal=causal, return_lse=True)
            sc.attention_backward(q, q, q, q, out, torch.zeros_like(lse), off, causal=causal)
        sc.group_norm(q.reshape(n, h * d), 2, offsets=off)
    torch.cuda.synchronize()
    assert torch.equal(wide, before)


@gpu
@pytest.mark.parametrize("causal", [False, True])
def test_attention_over_caches_with_room(dev, causal):
    """k_lengths: only the first rows of each item's keys count, whatever the others
    hold; lengths past the item's rows are cut, negative ones are none."""
    sc = _sc()
    h, hk, d, room = 8, 2, 64, 300
    used = [300, 1, 0, 128, 299, 1000, -5, 65]
    items = len(used)
    q = _randn((2 * items, h, d), torch.bfloat16, dev, 1)
    k, v = (_randn((items * room, hk, d), torch.bfloat16, dev, s) for s in (2, 3))
    off, koff = _offsets([2] * items, dev), _offsets([room] * items, dev)
    full = [min(max(u, 0), room) for u in used]
    for i, u in enumerate(full):
        k[i * room + u:(i + 1) * room] = float("nan")
        v[i * room + u:(i + 1) * room] = float("inf")
    lens = torch.tensor(used, dtype=torch.int32, device=dev)
    out, lse = sc.attention(q, k, v, off, koff, lens, causal=causal, return_lse=True)
    qn, kn, vn = _clean(q), _clean(k), _clean(v)
    args = (d ** -0.5, causal, off.tolist(), koff.tolist(), full)
    ro, rl = op.attention(qn, kn, vn, *args)
    do = _randn((2 * items, h, d), torch.bfloat16, dev, 4)
    to, tl, tq, tk, tv = _bounds(qn, kn, vn, _np(out), _np(do), *args, torch.bfloat16)
    _check(out, ro, to + 2.0 ** -8 * np.abs(ro), "out")
    _check(lse, rl, tl, "lse")
    grads = sc.attention_backward(do, q, k, v, out, lse, off, koff, lens, causal=causal)
    refs = op.attention_backward(_np(do), qn, kn, vn, _np(out), *args)
    for got, ref, tol, what in zip(grads, refs, (tq, tk, tv), ("grad_q", "grad_k", "grad_v")):
        _check(got, ref, tol + 2.0 ** -8 * np.abs(ref), what)  # zeros where nothing is used


# Walks long and rows few enough that two groups of waves share a workgroup's keys.
# rows per item, keys per item, heads, key heads, columns, causal
PAIRED = [
    ([1300, 1, 1700], [1345, 70, 1410], 2, 2, 64, False),  # 22, 2 and 23 tiles of keys
    ([1300, 0, 1700], [1280, 9, 1473], 4, 2, 128, True),
    ([1500], [1473], 2, 2, 32, False), ([900, 700], [1700, 1400], 4, 4, 96, True),
    ([1100], [6011], 2, 2, 128, False),                    # and in several runs
    ([700, 500, 600], [0, 5000, 64], 2, 1, 72, False),     # an item without keys, one of one tile
    ([1800], [1000], 4, 4, 64, True),                      # rows that see nothing
]


@gpu
@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("case", range(len(PAIRED)))
def test_attention_of_two_groups_of_waves(dev, case, dtype):
    sc = _sc()
    lengths, keys, h, hk, d, causal = PAIRED[case]
    n, nk = sum(lengths) + 2, sum(keys) + 3
    q = _randn((n, h, d), dtype, dev, case, 1.3)
    k, v = _randn((nk, 2 * hk, d), dtype, dev, case + 1000, 1.3).split([hk, hk], 1)
    k[nk - 3:], v[nk - 3:] = float("nan"), float("inf")
    # maxima that come late: the last keys' scores are the largest
    k[: nk - 3] *= (torch.arange(nk - 3, device=dev)[:, None, None] * (2.0 / nk)).to(dtype)
    off, koff = _offsets(lengths, dev), _offsets(keys, dev)
    out, lse = sc.attention(q, k, v, off, koff, causal=causal, return_lse=True)
    for _ in range(2):
        again, l2 = sc.attention(q, k, v, off, koff, causal=causal, return_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, l2)
    args = (np.float64(np.float32(d ** -0.5)), causal, off.tolist(), koff.tolist())
    ro, rl = op.attention(_np(q), _clean(k), _clean(v), *args)
    to, tl = _bounds(_np(q), _clean(k), _clean(v), None, None, *args, None, dtype)[:2]
    _check(out, ro, to + U[dtype] * np.abs(ro) + TINY[dtype], "out")
    _check(lse, rl, tl, "lse")
    # a row of NaN is one, and its neighbours in the tile do not see it
    row = lengths[0] // 2
    q[row] = float("nan")
    bad, lbad = sc.attention(q, k, v, off, koff, causal=causal, return_lse=True)
    sees = koff[1].item() - max(lengths[0] - 1 - row, 0) > 0 if causal else keys[0] > 0
    assert torch.isnan(bad[row]).all() == sees and torch.isnan(lbad[row]).all() == sees
    bad[row], lbad[row] = out[row], lse[row]
    assert torch.equal(bad, out) and torch.equal(lbad, lse)


@gpu
@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
def test_attention_extreme_scores(dev, dtype):
    """Scores of thousands, of either sign and rising along the keys: the running
    maximum moves with every tile; a row's weights end on one key."""
    sc = _sc()
    n, d = 400, 64
    q = torch.zeros((n, 2, d))
    k = torch.zeros((n, 2, d))
    q[:, 0, 0], q[:, 1, 0] = 100.0, -100.0
    k[:, :, 0] = torch.arange(n)[:, None] / 4.0
    q, k = q.to(dtype).to(dev), k.to(dtype).to(dev)
    v = _randn((n, 2, d), dtype, dev, 3)
    out, lse = sc.attention(q, k, v, scale=1.0, return_lse=True)
    ro, rl = op.attention(_np(q), _np(k), _np(v), 1.0, False)
    # scores are exact here (one product each); neighbours differ by 25, or by more where the type cannot hold k
    _check(lse, rl, 16 * V * np.abs(rl) + 1e-5, "lse")
    to = _bounds(_np(q), _np(k), _np(v), None, None, 1.0, False, None, None, None, dtype)[0]
    _check(out, ro, to + U[dtype] * np.abs(ro) + TINY[dtype], "out")


@gpu
def test_attention_gradients_of_small_size_in_fp16(dev):
    """Many keys and small incoming gradients: weights near 2^-13 and score gradients
    near 2^-27, below fp16's smallest numbers, keep their digits. The gradients are
    linear in grad_out, so those of grad_out 2^-9 are 2^-9 of grad_out's up to the
    roundings to subnormal results (2^-25 each) and of the ranges' powers of two."""
    sc = _sc()
    n, d = 8192, 64
    q, k, v = (_randn((n, 1, d), torch.float16, dev, s, 0.3) for s in (1, 2, 3))
    out, lse = sc.attention(q, k, v, return_lse=True)
    do = _randn((n, 1, d), torch.float16, dev, 4)
    small = (do.float() * 2.0 ** -9).half()
    do = (small.float() * 2.0 ** 9).half()  # the same digits
    big = sc.attention_backward(do, q, k, v, out, lse)
    low = sc.attention_backward(small, q, k, v, out, lse)
    ref = op.attention_backward(_np(do), _np(q), _np(k), _np(v), _np(out), d ** -0.5, False)
    tol = _bounds(_np(q), _np(k), _np(v), _np(out), _np(do), d ** -0.5, False, None, None, None, torch.float16)[2:]
    for a, b, r, t, what in zip(big, low, ref, tol, ("grad_q", "grad_k", "grad_v")):
        _check(a, r, t + 2.0 ** -11 * np.abs(r) + 2.0 ** -24, what)
        _check(b.double() * 512, r, t + 2.0 ** -11 * np.abs(r) + 2.0 ** -24 * 512, what + " of small ones")


@gpu
def test_attention_past_32_bit_offsets(dev):
    """A cache of more than 2^31 elements: the last item's rows, forward and backward."""
    sc = _sc()
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    n, d = (2 ** 31) // 128 + 500, 128
    k = torch.zeros((n, 1, d), dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    last = 200
    k[n - last:], v[n - last:] = (_randn((last, 1, d), torch.bfloat16, dev, s) for s in (1, 2))
    koff = torch.tensor([0, n - last, n], dtype=torch.int32, device=dev)
    q, off = _randn((3, 2, d), torch.bfloat16, dev, 3), torch.tensor([0, 1, 3], dtype=torch.int32, device=dev)
    out, lse = sc.attention(q, k, v, off, koff, causal=True, return_lse=True)
    assert not out[0].any()
    assert torch.allclose(lse[0].double().cpu(), torch.tensor(float(np.log(n - last))).double(), atol=1e-4)
    do = _randn((3, 2, d), torch.bfloat16, dev, 4)
    dq, dk, dv = sc.attention_backward(do, q, k, v, out, lse, off, koff, causal=True)
    qn, kn, vn, on, dn = _np(q[1:]), _np(k[n - last:]), _np(v[n - last:]), _np(out[1:]), _np(do[1:])
    to, _, tq, tk, tv = _bounds(qn, kn, vn, on, dn, d ** -0.5, True, None, [0, last], None, torch.bfloat16)
    ro, _ = op.attention(qn, kn, vn, d ** -0.5, True, None, [0, last])
    refs = op.attention_backward(dn, qn, kn, vn, on, d ** -0.5, True, None, [0, last])
    _check(out[1:], ro, to + 2.0 ** -8 * np.abs(ro), "out")
    for got, ref, tol, what in ((dq[1:], refs[0], tq, "grad_q"), (dk[n - last:], refs[1], tk, "grad_k"),
                                (dv[n - last:], refs[2], tv, "grad_v")):
        _check(got, ref, tol + 2.0 ** -8 * np.abs(ref), what)


@gpu
def test_group_norm_past_32_bit_offsets(dev):
    sc = _sc()
    c, last = 1024, 300
    n = (2 ** 31) // c + 2000
    x = torch.zeros((n, c), dtype=torch.float16, device=dev)
    x[n - last:] = _randn((last, c), torch.float16, dev, 1, 1.0, 0.5)
    off = torch.tensor([0, n - last, n], dtype=torch.int32, device=dev)
    y, mean, rstd = sc.group_norm(x, 32, act="silu", offsets=off, return_stats=True)
    alone = sc.group_norm(x[n - last:].clone(), 32, act="silu")
    assert not y[:n - last].any()
    # the same item on another path: statistics differ by their joining, (300 / 4 + 340) v
    _check(y[n - last:], _np(alone), 1e-4 * (1 + np.abs(_np(alone))) + 2.0 ** -10 * np.abs(_np(alone)), "y")
    g = _randn((last, c), torch.float16, dev, 2)
    dy = torch.zeros_like(x)
    dy[n - last:] = g
    gx, gw, gb = sc.group_norm_backward(dy, x, mean, rstd, act="silu", offsets=off)
    rx, rw, rb = sc.group_norm_backward(g, x[n - last:].clone(), mean[1:].clone(), rstd[1:].clone(), act="silu")
    assert not gx[:n - last].any()
    _check(gx[n - last:], _np(rx), 1e-4 + 2.0 ** -10 * np.abs(_np(rx)), "grad_x")
    _check(gw, _np(rw), 1e-4 * (1 + np.abs(_np(rw))), "grad_weight")
    _check(gb, _np(rb), 1e-4 * (1 + np.abs(_np(rb))), "grad_bias")


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------


def _all_of(sc, x, off, at, f, w):
    """One pass of every operator, forward and backward: a list of tensors."""
    y, mean, rstd = sc.group_norm(x, 8, w, w, act="silu", offsets=off, return_stats=True)
    rows = sc.rotary(y.view(-1, 4, 32), at, f)
    out, lse = sc.attention(rows[:, :2], rows[:, 2:3], rows[:, 3:], off, causal=True, return_lse=True)
    grads = sc.attention_backward(out, rows[:, :2], rows[:, 2:3], rows[:, 3:], out, lse, off, causal=True)
    gn = sc.group_norm_backward(y, x, mean, rstd, w, w, "silu", off)
    return [y, mean, rstd, rows, out, lse, *grads, *gn]


@gpu
@pytest.mark.parametrize("lengths", [[30, 0, 50], [1500, 2700]])
def test_graphs_and_streams(dev, lengths):
    """Two captured graphs, replayed in turn with eager work between them, give what
    eager calls give; so does another stream."""
    sc = _sc()
    n = sum(lengths)
    off, at = _offsets(lengths, dev), torch.arange(n, dtype=torch.int32, device=dev)
    f, w = sc.rotary_frequencies(32, device=dev), torch.linspace(0.5, 1.5, 128, device=dev)
    xs = [_randn((n, 128), torch.float16, dev, s) for s in range(4)]
    want = [[t.clone() for t in _all_of(sc, x, off, at, f, w)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all_of(sc, xs[0], off, at, f, w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs = []
    for _ in range(2):
        x = xs[0].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = _all_of(sc, x, off, at, f, w)
        graphs.append((g, x, res))
    for turn in range(6):
        g, x, res = graphs[turn % 2]
        x.copy_(xs[turn % 4])
        g.replay()
        eager = _all_of(sc, xs[3], off, at, f, w)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want[turn % 4])), turn
        assert all(torch.equal(a, b) for a, b in zip(eager, want[3])), turn
