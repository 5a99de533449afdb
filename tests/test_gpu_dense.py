"""The dense layers on the GPU (layer norm, linear, gated feed-forward, forward
and backward) against the fp64 oracle, on the very inputs the GPU reads.

Tolerances, per element, from the roundings that are made (u the unit roundoff
of the stored type: 2^-11 fp16, 2^-8 bf16, 2^-24 fp32; v = 2^-24):
- one rounding of a stored value: u |ref| (and 2^-24 for fp16 subnormals);
- an operand rounded to 16 bits between two products (h, dg, du, dz) carries
  u |operand|, which the next product turns into u sum |operand| |W|;
- an fp32 sum of K products: at most (K + 4) v sum |a| |b|;
- an fp32 activation: exp, reciprocal and erf are good to a few v, so value
  and slope are within 32 v (1 + |z|); a slope of at most 1.2 passes on the
  error of z;
- fp32 row statistics of C values: (C + 8) v relative to the terms summed.
Every bound is the sum of such terms; none is fitted.
"""
import numpy as np
import pytest
import torch

from oracle import dense as od

gpu = pytest.mark.gpu
V = 2.0 ** -24
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: V}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 1e-30, torch.float32: 1e-30}


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


def _check(got, ref, tol, what):
    got = _np(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300)):.3g} x the bound")


class Maker:
    """Seeded tensors; rows of a wider tensor full of NaN where pad > 0."""

    def __init__(self, dev, seed):
        self.dev, self.g = dev, torch.Generator().manual_seed(seed)

    def rows(self, n, c, dtype, pad=0, shift=0.0, scale=1.0):
        t = torch.full((n, c + 2 * pad), float("nan"), dtype=dtype)
        t[:, pad:pad + c] = (torch.randn((n, c), generator=self.g) * scale + shift).to(dtype)
        return t.to(self.dev)[:, pad:pad + c]

    def vec(self, c, shift=0.0):
        return (torch.randn((c,), generator=self.g) * 0.3 + shift).to(self.dev)

    def mat(self, k, n, dtype):
        return (torch.randn((k, n), generator=self.g) * k ** -0.5).to(dtype).to(self.dev)


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

NORM_SHAPES = [(1, 1, 0), (3, 7, 0), (0, 64, 0), (1, 1024, 0), (130, 64, 0), (257, 128, 0), (33, 100, 3),
               (129, 256, 8), (70, 515, 1), (65, 768, 0), (19, 1021, 0), (9, 2048, 0), (5, 2056, 0), (7, 5000, 0),
               (3, 4097, 1), (2, 8192, 0), (40, 32, 4), (5000, 48, 0)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,c,pad", NORM_SHAPES)
def test_layer_norm(dev, n, c, pad, dtype):
    sc = _sc()
    mk = Maker(dev, 1000 * n + c)
    affine = n != 33
    x = mk.rows(n, c, dtype, pad, shift=0.7, scale=1.3)
    w, b = (mk.vec(c, 1.0), mk.vec(c)) if affine else (None, None)
    eps = 1e-5
    y, mean, rstd = sc.layer_norm(x, w, b, eps=eps, return_stats=True)
    xn, wn, bn = _np(x), None if w is None else _np(w), None if b is None else _np(b)
    if n == 0:
        assert y.shape == (0, c) and mean.shape == (0,)
    else:
        ry, rm, rr = od.layer_norm(xn, wn, bn, eps)
        u = U[dtype]
        e = (c + 8) * V
        em = e * np.abs(xn).mean(1)  # error of the mean
        var = 1 / rr ** 2
        sd = np.sqrt(((xn - rm[:, None]) ** 2).mean(1))
        er = rr * (e + (2 * em * sd + em * em) / var)  # and of 1 / sqrt(var + eps)
        _check(mean, rm, em + V * np.abs(rm), "mean")
        _check(rstd, rr, er, "rstd")
        a = np.abs(xn - rm[:, None]) + V * (np.abs(xn) + np.abs(rm[:, None]))
        w1 = 1.0 if wn is None else np.abs(wn)
        b1 = 0.0 if bn is None else np.abs(bn)
        tol = w1 * (a * er[:, None] + rr[:, None] * (em[:, None] + V * (np.abs(xn) + np.abs(rm[:, None])))
                    + 4 * V * a * rr[:, None]) + 4 * V * b1 + u * np.abs(ry) + TINY[dtype]
        _check(y, ry, tol, "y")
    # gradients, for the statistics that the forward wrote
    dy = mk.rows(n, c, dtype, pad)
    gx, gw, gb = sc.layer_norm_backward(dy, x, mean, rstd, w)
    dyn, mn, rn = _np(dy), _np(mean), _np(rstd)
    rx, rw, rb = od.layer_norm_backward(dyn, xn, mn, rn, wn) if n else (np.zeros((0, c)), np.zeros(c), np.zeros(c))
    xh = (xn - mn[:, None]) * rn[:, None]
    exh = 4 * V * (np.abs(xn) + np.abs(mn[:, None])) * rn[:, None] + 4 * V * np.abs(xh)
    ad = np.abs(dyn) * (1.0 if wn is None else np.abs(wn))
    if n:
        s1 = ad.mean(1, keepdims=True)
        s2 = (ad * np.abs(xh)).mean(1, keepdims=True)
        es2 = (c + 8) * V * s2 + (ad * exh).mean(1, keepdims=True)
        tol = rn[:, None] * (8 * V * (ad + s1 + np.abs(xh) * s2) + (c + 8) * V * s1 + np.abs(xh) * es2 + exh * s2)
        _check(gx, rx, tol + U[dtype] * np.abs(rx) + TINY[dtype], "grad_x")
    _check(gw, rw, (n + 8) * V * (np.abs(dyn * xh)).sum(0) + (np.abs(dyn) * exh).sum(0) + 1e-30, "grad_weight")
    _check(gb, rb, (n + 8) * V * np.abs(dyn).sum(0) + 1e-30, "grad_bias")


@gpu
def test_layer_norm_far_from_zero_and_constant_rows(dev):
    """A mean of 1000 standard deviations keeps its variance (no difference
    of large squares); a constant row has variance 0 and y = bias."""
    sc = _sc()
    x = torch.randn((64, 256), generator=torch.Generator().manual_seed(5)) + 1000.0
    x[7] = 3.0
    b = torch.linspace(-1, 1, 256)
    y, _, rstd = sc.layer_norm(x.to(dev), None, b.to(dev), return_stats=True)
    ry, _, rr = od.layer_norm(x.numpy(), None, b.numpy(), 1e-5)
    # the mean's rounding (256 + 8) v 1000 moves a value of size 4 by 0.016 at most
    _check(y, ry, 0.02 + 0.02 * np.abs(ry), "y")
    assert torch.equal(y[7].cpu(), b)
    assert abs(float(rstd[7]) * np.sqrt(1e-5) - 1) < 1e-6


@gpu
def test_layer_norm_differences(dev):
    """grad_x against differences of the fp32 forward along random directions:
    step 2^-6 gives a truncation error of order 1e-4 and a rounding error of
    about 1e-6 sqrt(n c) / step, of directional derivatives near sqrt(n c)."""
    sc = _sc()
    g = torch.Generator().manual_seed(9)
    n, c = 50, 96
    x, dy, p = (torch.randn((n, c), generator=g).to(dev) for _ in range(3))
    w, b = torch.randn(c, generator=g).to(dev), torch.randn(c, generator=g).to(dev)
    _, m, r = sc.layer_norm(x, w, b, return_stats=True)
    gx, _, _ = sc.layer_norm_backward(dy, x, m, r, w)
    t = 2.0 ** -6
    up, down = (float((sc.layer_norm(x + s * t * p, w, b).double() * dy.double()).sum()) for s in (1, -1))
    got = float((gx.double() * p.double()).sum())
    assert abs(got - (up - down) / (2 * t)) < 0.02 * (n * c) ** 0.5


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------

LINEAR_SHAPES = [(1, 256, 1024, 0), (8, 40, 24, 1), (9, 40, 24, 1), (3, 2500, 40, 0), (4, 16, 8200, 0), (6, 24, 3000, 3),
                  (1, 1, 1, 0), (0, 16, 8, 0), (2, 8, 8, 0), (7, 72, 40, 0), (5, 33, 130, 1),
                 (16, 64, 64, 8), (127, 64, 128, 0), (128, 128, 128, 0), (129, 136, 264, 0), (300, 195, 77, 5),
                 (1000, 64, 512, 0), (513, 1000, 24, 0), (260, 512, 520, 4), (33, 2048, 96, 0)]


def _linear_tol(xn, Wn, bn, z, out, u, tiny, res=None):
    k = xn.shape[1]
    s = np.abs(xn) @ np.abs(Wn) + (0 if bn is None else np.abs(bn))
    ez = (k + 4) * V * s
    tol = 1.2 * ez + 32 * V * (1 + np.abs(z)) + u * np.abs(out) + tiny
    return (tol if res is None else tol + 2 * V * np.abs(res)), ez


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("shape", LINEAR_SHAPES, ids=str)
def test_linear(dev, shape, dtype):
    sc = _sc()
    n, cin, cout, pad = shape
    act = od.ACTS[(n + cin) % len(od.ACTS)]
    mk = Maker(dev, n * 7 + cin)
    x, W = mk.rows(n, cin, dtype, pad), mk.mat(cin, cout, dtype)
    bias = mk.vec(cout) if n != 128 else None
    res = mk.rows(n, cout, dtype, pad) if n % 2 else None
    u, tiny = U[dtype], TINY[dtype]
    out, pre = sc.linear(x, W, bias, act=act, residual=res, return_pre=True)
    same = sc.linear(x, W, bias, act=act, residual=res)
    assert torch.equal(out.view(torch.int16), same.view(torch.int16))
    xn, Wn, bn = _np(x), _np(W), None if bias is None else _np(bias)
    rn = None if res is None else _np(res)
    ro, rz = od.linear(xn, Wn, bn, act, rn)
    tol, ez = _linear_tol(xn, Wn, bn, rz, ro, u, tiny, rn)
    _check(pre, rz, ez + u * np.abs(rz) + tiny, "pre")
    _check(out, ro, tol, "out")
    # gradients, for the pre-activation that the forward wrote
    dy = mk.rows(n, cout, dtype, pad)
    gx, gw, gb = sc.linear_backward(dy, x, W, pre if act != "none" else None, act=act)
    dyn, zn = _np(dy), _np(pre)
    rx, rw, rb, dz = od.linear_backward(dyn, xn, Wn, zn, act)
    ed = np.abs(dyn) * 32 * V * (1 + np.abs(zn)) if act != "none" else 0 * dyn  # dz before rounding
    er = ed + (u * np.abs(dz) + tiny if act != "none" else 0)                    # and after
    aW, ax, ad = np.abs(Wn), np.abs(xn), np.abs(dz)
    _check(gx, rx, er @ aW.T + (cout + 4) * V * (ad @ aW.T) + u * np.abs(rx) + tiny, "grad_x")
    _check(gw, rw, ax.T @ er + (n + 4) * V * (ax.T @ ad) + u * np.abs(rw) + tiny, "grad_W")
    _check(gb, rb, ed.sum(0) + (n + 8) * V * ad.sum(0) + 1e-30, "grad_b")
    again = sc.linear_backward(dy, x, W, pre if act != "none" else None, act=act)
    assert all(torch.equal(a, b) for a, b in zip((gx, gw, gb), again))


@gpu
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("cout", [255, 257, 1030, 8191, 8193])
def test_linear_few_rows(dev, rows, cout):
    """Every width of strip for every count of rows, with a k that no strip's
    threads divide and rows of W that start anywhere."""
    sc = _sc()
    cin = 131
    mk = Maker(dev, rows * 7 + cout)
    for dtype in (torch.float16, torch.bfloat16):
        x, W, bias = mk.rows(rows, cin, dtype, 3), mk.mat(cin, cout, dtype), mk.vec(cout)
        out = sc.linear(x, W, bias, act="silu")
        xn, Wn, bn = _np(x), _np(W), _np(bias)
        ro, rz = od.linear(xn, Wn, bn, "silu", None)
        _check(out, ro, _linear_tol(xn, Wn, bn, rz, ro, U[dtype], TINY[dtype])[0], "out")


@gpu
def test_wide_tiles(dev):
    """Products large enough for the 256 x 256 tile, in both orders of the weight,
    of plain and of blocked rows, against torch in fp64 on some rows of the
    result (rows at both ends and inside, all columns)."""
    sc = _sc()
    n, cin, cout = 66001, 512, 520
    mk = Maker(dev, 2)
    x, W, dy = mk.rows(n, cin, torch.bfloat16), mk.mat(cin, cout, torch.bfloat16), mk.rows(n, cout, torch.bfloat16)
    b = mk.vec(cout)
    out, pre = sc.linear(x, W, b, act="silu", return_pre=True)
    at = torch.tensor([0, 1, 127, 128, 255, 256, 33000, n - 130, n - 2, n - 1], device=dev)
    z = x[at].double() @ W.double() + b.double()
    s = x[at].double().abs() @ W.double().abs() + b.double().abs()
    ez = (cin + 4) * V * s
    u = U[torch.bfloat16]
    _check(pre[at], z.cpu().numpy(), (ez + u * z.abs()).cpu().numpy() + 1e-30, "pre")
    r = torch.nn.functional.silu(z)
    _check(out[at], r.cpu().numpy(), (1.2 * ez + 32 * V * (1 + z.abs()) + u * r.abs()).cpu().numpy(), "out")
    for act, p in ((None, None), ("silu", pre)):
        gx = sc.linear_backward(dy, x, W, p, act=act, needs=(True, False, False))[0]
        dz = dy[at].double()
        ed = torch.zeros_like(dz)
        if act:
            v, d = od.act(pre[at].double().cpu().numpy(), act)
            ed = dz.abs() * 32 * V * (1 + pre[at].double().abs())
            dz = dz * torch.from_numpy(d).to(dev)
            ed = ed + u * dz.abs()
        rx, sx = dz @ W.double().t(), dz.abs() @ W.double().abs().t()
        tol = ed @ W.double().abs().t() + (cout + 4) * V * sx + u * rx.abs() + 1e-30
        _check(gx[at], rx.cpu().numpy(), tol.cpu().numpy(), f"grad_x {act}")


@gpu
def test_offsets_past_32_bits(dev):
    """17 million sites: pre-activations, dz and norm rows of more than 2^31
    elements. Rows at both ends and around element 2^31 against the oracle on
    those rows alone; a NaN tail row would show reads past the end."""
    sc = _sc()
    n, c, f = 17_000_000, 16, 64
    g = torch.Generator(device=dev).manual_seed(1)
    half = torch.float16
    x = torch.randn((n, c), generator=g, device=dev).to(half)
    Wi = (torch.randn((c, 2 * f), generator=g, device=dev) * c ** -0.5).to(half)
    Wo = (torch.randn((f, c), generator=g, device=dev) * f ** -0.5).to(half)
    edge = 2 ** 31 // (2 * f)
    at = torch.tensor([0, 1, edge - 1, edge, edge + 1, n - 129, n - 2, n - 1], device=dev)
    u, tiny = U[half], TINY[half]
    out, pre = sc.gated_ffn(x, Wi, None, Wo, act="silu", return_pre=True)
    xn, wi, wo = _np(x[at]), _np(Wi), _np(Wo)
    ro, rz, h = od.gated_ffn(xn, wi, None, wo, None, "silu", None)
    ez = (c + 4) * V * (np.abs(xn) @ np.abs(wi))
    _check(pre[at], rz, ez + u * np.abs(rz) + tiny, "pre")
    eh = (1.2 * ez[:, :f] + 32 * V * (1 + np.abs(rz[:, :f]))) * (np.abs(rz[:, f:]) + ez[:, f:]) \
        + np.abs(rz[:, :f]) * ez[:, f:] + (4 * V + u) * np.abs(h) + tiny
    _check(out[at], ro, eh @ np.abs(wo) + (f + 4) * V * (np.abs(h) @ np.abs(wo)) + u * np.abs(ro) + tiny, "out")
    gx, _, _, gwo, gb = sc.gated_ffn_backward(out, x, Wi, Wo, pre, act="silu")
    dyn, zn = _np(out[at]), _np(pre[at])
    rx, _, _, _, _, dz, _ = od.gated_ffn_backward(dyn, xn, wi, wo, zn, "silu")
    adh = np.abs(dyn) @ np.abs(wo).T
    a, d = od.act(zn[:, :f], "silu")
    eact = 32 * V * (1 + np.abs(zn[:, :f]))
    edh = (c + 4) * V * adh
    ed = np.concatenate([(edh * np.abs(d) + adh * eact) * np.abs(zn[:, f:]), edh * np.abs(a) + adh * eact], 1)
    er = ed + (4 * V + u) * np.abs(dz) + tiny
    _check(gx[at], rx, er @ np.abs(wi).T + (2 * f + 4) * V * (np.abs(dz) @ np.abs(wi).T) + u * np.abs(rx) + tiny, "grad_x")
    # the weight gradient's sums of 17 million terms, against torch in fp64;
    # many are past fp16's largest number, which has to give infinities
    p64, u64 = pre[:, :f].double(), pre[:, f:].double()
    h64, dy64 = torch.nn.functional.silu(p64) * u64, out.double()
    ref = h64.t() @ dy64
    eh = (u + 4 * V) * h64.abs() + 32 * V * (1 + p64.abs()) * u64.abs() + tiny
    tol = eh.t() @ dy64.abs() + (n / 256 + 260) * V * (h64.abs().t() @ dy64.abs()) + u * ref.abs()
    del p64, u64, h64, dy64, eh
    inside, beyond = ref.abs() + tol < 65504, ref.abs() - tol > 65520
    assert bool((((gwo.double() - ref).abs() <= tol) | ~inside).all())
    assert bool(((gwo.double() == torch.sign(ref) * float("inf")) | ~beyond).all())
    # the column sum: n terms in fp32, against torch in fp64
    ref = out.double().sum(0)
    tol = (n / 1024 + 2000) * V * out.double().abs().sum(0)  # 1024 runs, then their sums
    assert bool(((gb.double() - ref).abs() <= tol).all())
    del gx, gwo, dz
    y, mean, rstd = sc.layer_norm(pre, return_stats=True)
    ry, _, rr = od.layer_norm(zn, None, None, 1e-5)
    _check(y[at], ry, 64 * (2 * f + 8) * V * (1 + np.abs(ry)) + u * np.abs(ry) + tiny, "norm")
    del y
    gx, _, _ = sc.layer_norm_backward(pre, pre, mean, rstd)
    rx, _, _ = od.layer_norm_backward(zn, zn, _np(mean[at]), _np(rstd[at]), None)
    # d - mean(d) - xh mean(d xh) of d = x cancels to eps: the terms' size counts
    _check(gx[at], rx, 64 * (2 * f + 8) * V * (1 + np.abs(zn)) * rr[:, None] ** 2 * (1 + np.abs(zn)) ** 2 + u * np.abs(rx) + tiny,
           "norm grad")


@gpu
@pytest.mark.parametrize("act", od.ACTS)
def test_linear_every_activation(dev, act):
    """Every activation's value and slope over pre-activations from -30 to 30
    (an identity weight puts them there exactly)."""
    sc = _sc()
    c = 64
    x = torch.linspace(-30, 30, 64 * c).reshape(64, c).to(torch.float16).to(dev)
    W = torch.eye(c, dtype=torch.float16, device=dev)
    out, pre = sc.linear(x, W, None, act=act, return_pre=True)
    assert torch.equal(pre, x)
    xn = _np(x)
    v, d = od.act(xn, act)
    _check(out, v, 32 * V * (1 + np.abs(xn)) + 2.0 ** -11 * np.abs(v) + 2.0 ** -24, "value")
    one = torch.ones_like(x)
    gx, _, gb = sc.linear_backward(one, x, W, pre, act=act)
    tol = 32 * V * (1 + np.abs(xn))
    _check(gx, d, tol + 2 * 2.0 ** -11 * np.abs(d) + 2.0 ** -23, "slope")
    _check(gb, d.sum(0), tol.sum(0) + 72 * V * np.abs(d).sum(0), "sum of slopes")


@gpu
def test_linear_rows_of_nan_and_infinity_stay_their_own(dev):
    """A NaN or an infinity reaches its own row alone, in every product that
    does not sum over rows."""
    sc = _sc()
    mk = Maker(dev, 77)
    n, cin, cout = 200, 72, 136
    x, W, b = mk.rows(n, cin, torch.float16), mk.mat(cin, cout, torch.float16), mk.vec(cout)
    clean = sc.linear(x, W, b, act="relu")
    y = x.clone()
    y[5, 3], y[130, 71], y[199, 0] = float("nan"), float("inf"), float("-inf")
    out = sc.linear(y, W, b, act="relu")
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[[5, 130, 199]] = False
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[5]).all())
    assert not bool(torch.isfinite(out[130]).all())


@gpu
def test_linear_writes_nothing_else(dev):
    """The C entry points write their outputs' elements alone: canaries around
    every output survive, at widths that are read through copies and not."""
    sc = _sc()
    lib = sc.load_library()
    for n, cin, cout in ((5, 33, 77), (130, 64, 128), (257, 40, 72)):
        mk = Maker(dev, n)
        x, W, b = mk.rows(n, cin, torch.float16), mk.mat(cin, cout, torch.float16), mk.vec(cout)
        pad = 64
        buf = torch.full((2, n * cout + 2 * pad), 7.0, dtype=torch.float16, device=dev)
        out, pre = buf[0, pad:], buf[1, pad:]
        nb = lib.submconv_linear_workspace_bytes(n, cin, cout, 0)
        ws = torch.empty(nb + 256, dtype=torch.uint8, device=dev)
        ws[nb:] = 9
        sc._check(lib.submconv_linear(sc._ptr(x), cin, n, sc._ptr(W), sc._ptr(b), None, 0, sc._ptr(out),
                                      sc._ptr(pre), cin, cout, 2, 0, sc._ptr(ws), nb, sc._stream(dev)))
        assert bool((buf[:, :pad] == 7).all()) and bool((buf[:, pad + n * cout:] == 7).all())
        assert bool((ws[nb:] == 9).all())
        ro, rp = sc.linear(x, W, b, act="silu", return_pre=True)
        assert torch.equal(out[:n * cout].reshape(n, cout), ro)
        assert torch.equal(pre[:n * cout].reshape(n, cout), rp)


# ---------------------------------------------------------------------------
# gated feed-forward
# ---------------------------------------------------------------------------

FFN_SHAPES = [(257, 65, 65, 128, 0), (600, 128, 200, 9, 1), (300, 16, 130, 64, 0), (520, 120, 33, 127, 0),
              (1, 64, 128, 64, 0), (8, 33, 1100, 17, 2), (5, 16, 3000, 24, 0), (1, 512, 2048, 512, 0), (0, 32, 64, 16, 0), (2, 16, 8, 8, 0), (3, 9, 5, 3, 1),
              (9, 40, 100, 24, 0), (64, 64, 64, 64, 0), (130, 128, 512, 128, 0), (129, 100, 267, 100, 0),
              (300, 72, 136, 200, 8), (1000, 64, 256, 64, 3), (257, 256, 72, 136, 0)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("shape", FFN_SHAPES, ids=str)
def test_gated_ffn(dev, shape, dtype):
    sc = _sc()
    n, cin, F, cout, pad = shape
    act = od.ACTS[(n + F) % len(od.ACTS)]
    mk = Maker(dev, n * 11 + F)
    x, Wi, Wo = mk.rows(n, cin, dtype, pad), mk.mat(cin, 2 * F, dtype), mk.mat(F, cout, dtype)
    bi, bo = (mk.vec(2 * F), mk.vec(cout)) if n != 64 else (None, None)
    res = mk.rows(n, cout, dtype, pad) if n % 2 else None
    u, tiny = U[dtype], TINY[dtype]
    out, pre = sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res, return_pre=True)
    # without pre-activations to write, narrow layers take another kernel
    alone = sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res)
    again = sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res)
    assert torch.equal(alone.view(torch.int16), again.view(torch.int16))
    xn, Win, Won = _np(x), _np(Wi), _np(Wo)
    bin_, bon = (None, None) if bi is None else (_np(bi), _np(bo))
    rn = None if res is None else _np(res)
    ro, rz, h = od.gated_ffn(xn, Win, bin_, Won, bon, act, rn)
    ez = (cin + 4) * V * (np.abs(xn) @ np.abs(Win) + (0 if bin_ is None else np.abs(bin_)))
    _check(pre, rz, ez + u * np.abs(rz) + tiny, "pre")
    g, up = rz[:, :F], rz[:, F:]
    a, _ = od.act(g, act)
    ea = 1.2 * ez[:, :F] + 32 * V * (1 + np.abs(g))
    eh = ea * (np.abs(up) + ez[:, F:]) + np.abs(a) * ez[:, F:] + 4 * V * np.abs(h) + u * np.abs(h) + tiny
    aWo = np.abs(Won)
    tol = eh @ aWo + (F + 4) * V * (np.abs(h) @ aWo + (0 if bon is None else np.abs(bon))) \
        + (0 if rn is None else 2 * V * np.abs(rn)) + u * np.abs(ro) + tiny
    _check(out, ro, tol, "out")
    _check(alone, ro, tol, "out without pre")
    # gradients, for the pre-activations that the forward wrote
    dy = mk.rows(n, cout, dtype, pad)
    grads = sc.gated_ffn_backward(dy, x, Wi, Wo, pre, act=act)
    dyn, zn = _np(dy), _np(pre)
    rx, rwi, rbi, rwo, rbo, dz, h = od.gated_ffn_backward(dyn, xn, Win, Won, zn, act)
    g, up = zn[:, :F], zn[:, F:]
    a, d = od.act(g, act)
    adh = np.abs(dyn) @ aWo.T
    edh = (cout + 4) * V * adh
    eact = 32 * V * (1 + np.abs(g))
    ed = np.concatenate([edh * np.abs(up * d) + adh * np.abs(up) * eact, edh * np.abs(a) + adh * eact], 1) \
        + 4 * V * np.abs(dz)
    er = ed + u * np.abs(dz) + tiny
    eh = eact * np.abs(up) + 4 * V * np.abs(h) + u * np.abs(h) + tiny
    aWi, ax, ad = np.abs(Win), np.abs(xn), np.abs(dz)
    _check(grads[0], rx, er @ aWi.T + (2 * F + 4) * V * (ad @ aWi.T) + u * np.abs(rx) + tiny, "grad_x")
    _check(grads[1], rwi, ax.T @ er + (n + 4) * V * (ax.T @ ad) + u * np.abs(rwi) + tiny, "grad_W_in")
    _check(grads[2], rbi, ed.sum(0) + (n + 8) * V * ad.sum(0) + 1e-30, "grad_b_in")
    _check(grads[3], rwo, eh.T @ np.abs(dyn) + (n + 4) * V * (np.abs(h).T @ np.abs(dyn)) + u * np.abs(rwo) + tiny,
           "grad_W_out")
    _check(grads[4], rbo, (n + 8) * V * np.abs(dyn).sum(0) + 1e-30, "grad_b_out")
    again = sc.gated_ffn_backward(dy, x, Wi, Wo, pre, act=act)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


@gpu
def test_gated_ffn_full_and_partial_rounds(dev):
    """The one-kernel block over a whole round of workgroups (65536 rows) and a
    part of the next, short and long: rows around the seam and at both ends
    against the oracle, the rows past it against the call on those alone, which
    gives a wave half as many rows (two roundings of h and one of out apart at
    most: 4 u of the largest)."""
    sc = _sc()
    for n, c, f in ((65536 + 77, 64, 96), (65536 + 40000, 48, 40), (65536, 128, 72)):
        mk = Maker(dev, n)
        x, Wi, Wo = mk.rows(n, c, torch.float16, 3), mk.mat(c, 2 * f, torch.float16), mk.mat(f, c, torch.float16)
        bi, bo = mk.vec(2 * f), mk.vec(c)
        out = sc.gated_ffn(x, Wi, bi, Wo, bo, act="gelu", residual=x)
        at = torch.tensor([i for i in (0, 1, 65534, 65535, 65536, 65537, n - 2, n - 1) if i < n], device=dev)
        xn, wi, wo, b1, b2 = _np(x[at]), _np(Wi), _np(Wo), _np(bi), _np(bo)
        ro, rz, h = od.gated_ffn(xn, wi, b1, wo, b2, "gelu", xn)
        u, tiny = U[torch.float16], TINY[torch.float16]
        ez = (c + 4) * V * (np.abs(xn) @ np.abs(wi) + np.abs(b1))
        g, up = rz[:, :f], rz[:, f:]
        eh = (1.2 * ez[:, :f] + 32 * V * (1 + np.abs(g))) * (np.abs(up) + ez[:, f:]) + np.abs(g) * ez[:, f:] \
            + (4 * V + u) * np.abs(h) + tiny
        tol = eh @ np.abs(wo) + (f + 4) * V * (np.abs(h) @ np.abs(wo) + np.abs(b2)) + 2 * V * np.abs(xn) \
            + u * np.abs(ro) + tiny
        _check(out[at], ro, tol, f"out {n}")
        tail = sc.gated_ffn(x[65536 - 64:], Wi, bi, Wo, bo, act="gelu", residual=x[65536 - 64:])
        err = float((out[65536 - 64:].float() - tail.float()).abs().max())
        assert err <= 4 * u * float(tail.float().abs().max()), (n, err)


@gpu
def test_gated_ffn_leaves_gradients_out(dev):
    sc = _sc()
    mk = Maker(dev, 31)
    x, Wi, Wo = mk.rows(70, 40, torch.float16), mk.mat(40, 48, torch.float16), mk.mat(24, 16, torch.float16)
    _, pre = sc.gated_ffn(x, Wi, None, Wo, return_pre=True)
    dy = mk.rows(70, 16, torch.float16)
    full = sc.gated_ffn_backward(dy, x, Wi, Wo, pre)
    for k in range(5):
        needs = tuple(j == k for j in range(5))
        part = sc.gated_ffn_backward(dy, x, Wi, Wo, pre, needs=needs)
        assert [p is not None for p in part] == list(needs)
        assert torch.equal(part[k], full[k])
    lin = sc.linear_backward(dy, mk.rows(70, 24, torch.float16), Wo, needs=(True, False, False))
    assert lin[1] is None and lin[2] is None


# ---------------------------------------------------------------------------
# modules, streams, graphs, refusals
# ---------------------------------------------------------------------------


@gpu
def test_modules_train_like_torch(dev):
    """The modules' gradients in fp16 against the same block of torch modules
    in fp64: relative 2-norm error within 1 % (a chain of six fp16 roundings of
    2^-11 each, amplified by cancellation in the norm's gradient by less than
    three)."""
    sc = _sc()
    torch.manual_seed(3)
    n, c, f = 333, 48, 80
    proj = sc.Linear(24, c, act="silu", device=dev)
    norm = sc.LayerNorm(c, device=dev)
    ffn = sc.GatedFeedForward(c, f, device=dev)
    x = torch.randn(n, 24, device=dev).half().requires_grad_()
    h = proj(x)
    out = ffn(norm(h), residual=h)
    dy = torch.randn_like(out)
    (out * dy).sum().backward()

    d = lambda t: t.detach().double().requires_grad_()  # noqa: E731
    px, pw, pb, nw, nb_, wi, bi, wo, bo = map(d, (x, proj.weight, proj.bias, norm.weight, norm.bias, ffn.w_in, ffn.b_in,
                                                  ffn.w_out, ffn.b_out))
    F = torch.nn.functional
    rh = F.silu(px @ pw + pb)
    z = F.layer_norm(rh, (c,), nw, nb_, 1e-5) @ wi + bi
    ro = (F.silu(z[:, :f]) * z[:, f:]) @ wo + bo + rh
    (ro * dy.double()).sum().backward()
    pairs = [(out, ro), (x.grad, px.grad), (proj.weight.grad, pw.grad), (proj.bias.grad, pb.grad),
             (norm.weight.grad, nw.grad), (norm.bias.grad, nb_.grad), (ffn.w_in.grad, wi.grad), (ffn.b_in.grad, bi.grad),
             (ffn.w_out.grad, wo.grad), (ffn.b_out.grad, bo.grad)]
    for i, (a, b) in enumerate(pairs):
        assert a.dtype in (torch.float16, torch.float32)
        err = float((a.detach().double() - b.detach()).norm() / b.detach().norm())
        assert err < 1e-2, (i, err)


@gpu
def test_gradients_of_expanded_and_scaled_losses(dev):
    """sum() hands the backward an expanded gradient; it counts as ones."""
    sc = _sc()
    ffn = sc.GatedFeedForward(16, 24, device=dev)
    x = torch.randn(40, 16, device=dev).half().requires_grad_()
    ffn(x).sum().backward()
    assert torch.equal(ffn.b_out.grad, torch.full((16,), 40.0, device=dev))


@gpu
def test_block_equals_torch(dev):
    """A residual block (projection, convolution, norm, gated feed-forward, skip
    connection) and all its gradients against torch in fp64 over the exported
    neighbour map: relative 2-norm error within 1 % (as for the modules: a chain
    of fp16 roundings of 2^-11, here eight)."""
    sc = _sc()
    torch.manual_seed(4)
    G, c, f = 12, 32, 72
    lin = torch.randperm(G ** 3)[:500].sort().values
    coords = torch.stack([0 * lin, lin // (G * G), lin // G % G, lin % G], 1).int().to(dev)
    kmap = sc.build_map(coords, (G, G, G), 1)
    block = sc.SparseConvBlock(c, f, cin=16, device=dev)
    x = torch.randn(500, 16, device=dev).half().requires_grad_()
    out = block(kmap, x)
    dy = torch.randn_like(out)
    (out * dy).sum().backward()
    with torch.no_grad():
        assert float((block(kmap, x) - out).abs().max()) <= 2 * 2.0 ** -11 * float(out.abs().max())

    p = {k: v.detach().double().requires_grad_() for k, v in block.named_parameters()}
    rx = x.detach().double().requires_grad_()
    F = torch.nn.functional
    h = F.silu(rx @ p["proj.weight"] + p["proj.bias"])
    nbr = kmap.export().long()
    rows = torch.cat([h, h.new_zeros(1, c)])[torch.where(nbr < 0, 500, nbr)]  # [N,27,C]
    conv = rows.reshape(500, 27 * c) @ p["conv_weight"].reshape(27 * c, c) + p["conv_bias"]
    z = F.layer_norm(conv, (c,), p["norm.weight"], p["norm.bias"], 1e-5) @ p["ffn.w_in"] + p["ffn.b_in"]
    ref = (F.silu(z[:, :f]) * z[:, f:]) @ p["ffn.w_out"] + p["ffn.b_out"] + h
    (ref * dy.double()).sum().backward()
    pairs = [("out", out, ref), ("x", x.grad, rx.grad)]
    pairs += [(k, v.grad, p[k].grad) for k, v in block.named_parameters()]
    for name, a, b in pairs:
        err = float((a.detach().double() - b.detach()).norm() / b.detach().norm())
        assert err < 1e-2, (name, err)
    kmap.free()


@gpu
def test_example_runs(dev):
    """The training example: every loss is finite and the last is the smallest
    of the first and last; the block runs without gradients afterwards."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, final = mod.train(grid=24, channels=32, steps=10)
    assert all(np.isfinite(losses)) and np.isfinite(final)
    assert losses[-1] < losses[0]


@gpu
def test_streams(dev):
    """The operators run on the current stream: chains on four streams at once
    equal the chain run alone."""
    sc = _sc()
    mk = Maker(dev, 8)
    Wi, Wo = mk.mat(64, 256, torch.float16), mk.mat(128, 64, torch.float16)
    xs = [mk.rows(5000 + 7 * i, 64, torch.float16) for i in range(4)]

    def chain(x):
        y, m, r = sc.layer_norm(x, return_stats=True)
        o, pre = sc.gated_ffn(y, Wi, None, Wo, residual=x, return_pre=True)
        g = sc.gated_ffn_backward(o, y, Wi, Wo, pre)
        return [o, *g, *sc.layer_norm_backward(g[0], x, m, r)]

    alone = [chain(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append(chain(x))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@gpu
def test_graph_replays(dev):
    """A captured forward and backward replays to the eager result, with eager
    work between the replays."""
    sc = _sc()
    mk = Maker(dev, 12)
    x, W = mk.rows(700, 72, torch.bfloat16), mk.mat(72, 40, torch.bfloat16)
    b, dy = mk.vec(40), mk.rows(700, 40, torch.bfloat16)

    def step():
        out, pre = sc.linear(x, W, b, act="gelu", return_pre=True)
        return [out, *sc.linear_backward(dy, x, W, pre, act="gelu")]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, ref)), k


@gpu
def test_refusals(dev):
    sc = _sc()
    h = dict(dtype=torch.float16, device=dev)
    x, W, b = torch.zeros((4, 8), **h), torch.zeros((8, 16), **h), torch.zeros(16, device=dev)
    bad = [
        (TypeError, lambda: sc.linear(x.float(), W, b)),
        (TypeError, lambda: sc.linear(x, W.bfloat16(), b)),
        (TypeError, lambda: sc.linear(x, W, b.half())),
        (ValueError, lambda: sc.linear(x.cpu(), W, b)),
        (ValueError, lambda: sc.linear(x, W.cpu(), b)),
        (ValueError, lambda: sc.linear(x, W[:7], b)),
        (ValueError, lambda: sc.linear(x, W, b[:15])),
        (ValueError, lambda: sc.linear(x, W.t().contiguous().t(), b)),
        (ValueError, lambda: sc.linear(x[:, ::2], W[:4], b)),
        (ValueError, lambda: sc.linear(x[:1].expand(4, 8), W, b)),
        (ValueError, lambda: sc.linear(x, W, b, act="tanh")),
        (ValueError, lambda: sc.linear(x, W, b, residual=torch.zeros((3, 16), **h))),
        (ValueError, lambda: sc.linear(x, W, b, residual=torch.zeros((4, 8), **h))),
        (TypeError, lambda: sc.linear_backward(torch.zeros((4, 16), **h), x, W, None, act="silu")),
        (ValueError, lambda: sc.linear_backward(torch.zeros((5, 16), **h), x, W)),
        (ValueError, lambda: sc.gated_ffn(x, W, None, torch.zeros((7, 8), **h))),
        (ValueError, lambda: sc.gated_ffn_backward(x, x, W, torch.zeros((8, 8), **h), torch.zeros((4, 15), **h))),
        (TypeError, lambda: sc.layer_norm(x.double())),
        (ValueError, lambda: sc.layer_norm(x[0])),
        (ValueError, lambda: sc.layer_norm(x, torch.zeros(7, device=dev))),
        (sc.SubmconvError, lambda: sc.layer_norm(torch.zeros((2, 8193), device=dev))),
        (sc.SubmconvError, lambda: sc.layer_norm(x, eps=-1.0)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was taken")
    # the C entry points: NULL, workspace, strides, kinds
    lib = sc.load_library()
    p, st = sc._ptr, sc._stream(dev)
    out = torch.zeros((4, 16), **h)
    args = [p(x), 8, 4, p(W), None, None, 0, p(out), None, 8, 16, 0, 0, None, 0, st]

    def call(**k):
        a = list(args)
        for i, v in k.items():
            a[int(i[1:])] = v
        return lib.submconv_linear(*a)

    assert call() == 0
    assert call(_0=None) == -1 and call(_3=None) == -1 and call(_7=None) == -1
    assert call(_1=7) == -1 and call(_1=1 << 40) == -4
    assert call(_9=0) == -4 and call(_11=9) == -1 and call(_12=2) == -1 and call(_2=-1) == -1
    odd, outs = torch.zeros(9 * 8 + 1, **h)[1:], torch.zeros((9, 16), **h)
    assert call(_0=p(odd)) == 0   # few rows are read as they are
    assert call(_0=p(odd), _2=9, _7=p(outs)) == -1  # more need a copy: workspace missing
    assert b"workspace" in lib.submconv_last_error()
    assert lib.submconv_linear_workspace_bytes(4, 0, 16, 0) == -4
    assert lib.submconv_gated_ffn_workspace_bytes(-1, 8, 16, 8, 0) == -1
    torch.cuda.synchronize()
