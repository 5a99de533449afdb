"""The dense layers at sizes that take each of their large kernels: the 128 x
128 tile of three buffers, the 256 x 256 tile, two-buffer gate kernels, 256 x
256 weight gradients of plain and blocked operands, and the one-kernel gated
block at both widths and both counts of rows a wave.

Most inputs are small whole numbers, chosen so that every product, sum and
rounding between two products is exact (whole numbers up to 256 in bf16, 2048 in
fp16, 2^24 in fp32): results then equal the fp64 value rounded once, bit for bit,
and one element missing, doubled or misplaced anywhere shows. Rows lie in a
wider and longer buffer full of NaN, which a read outside them would bring in.
"""
import numpy as np
import pytest
import torch

from oracle import dense as od

gpu = pytest.mark.gpu
V = 2.0 ** -24
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: V}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 1e-30, torch.float32: 1e-30}
TYPES = pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])


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


class Whole:
    """Seeded whole numbers on the device."""

    def __init__(self, dev, seed):
        self.dev, self.g = dev, torch.Generator(device=dev).manual_seed(seed)

    def _ints(self, shape, most):
        return torch.randint(-most, most + 1, shape, generator=self.g, device=self.dev)

    def rows(self, n, c, dtype, most, pad=0):
        """Rows between NaN columns (pad > 0) and NaN rows."""
        t = torch.full((n + 6, c + 2 * pad), float("nan"), dtype=dtype, device=self.dev)
        t[2:2 + n, pad:pad + c] = self._ints((n, c), most).to(dtype)
        return t[2:2 + n, pad:pad + c]

    def mat(self, k, n, dtype, most):
        return self._ints((k, n), most).to(dtype)

    def few(self, k, n, dtype, count):
        """A matrix with at most `count` entries of +-1 in each column."""
        t = torch.zeros((k, n), device=self.dev)
        at = torch.randint(0, k, (count, n), generator=self.g, device=self.dev)
        sign = torch.randint(0, 2, (count, n), generator=self.g, device=self.dev).float() * 2 - 1
        return t.scatter_(0, at, sign).to(dtype)

    def vec(self, c, most):
        return self._ints((c,), most).float()


def _same(got, ref, what):
    ref = ref.to(got.dtype)
    if not torch.equal(got, ref):
        bad = (got != ref) | got.isnan()
        at = bad.nonzero()[0].tolist()
        pytest.fail(f"{what}: {int(bad.sum())} of {bad.numel()} differ, the first at {at}: "
                    f"{float(got[tuple(at)])} for {float(ref[tuple(at)])}")


# 33001 x 136 -> 264: three buffers for the forward, for dx on plain rows (no
# activation) and blocked ones, 256 x 256 tiles for dW; 40001 x 72 -> 130:
# odd widths, through copies; 66001 x 512 -> 520: the 256 x 256 forward; the
# others few tiles, dx split over k, narrow weight gradients.
LINEAR = [(33001, 136, 264, 8), (33001, 136, 264, 0), (40001, 72, 130, 3), (66001, 512, 520, 0), (300, 200, 1030, 0),
          (9001, 128, 128, 0), (1000, 520, 1000, 5), (300, 200, 1032, 0)]


@gpu
@TYPES
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("shape", LINEAR, ids=str)
def test_linear_whole_numbers(dev, shape, act, dtype):
    sc = _sc()
    n, cin, cout, pad = shape
    mk = Whole(dev, n + cin)
    x, W, b = mk.rows(n, cin, dtype, 2, pad), mk.mat(cin, cout, dtype, 2), mk.vec(cout, 9)
    res = mk.rows(n, cout, dtype, 9, pad)
    out, pre = sc.linear(x, W, b, act=act, residual=res, return_pre=True)
    z = x.double() @ W.double() + b.double()
    _same(pre, z, "pre")
    _same(out, (z.clamp(min=0) if act == "relu" else z) + res.double(), "out")
    _same(sc.linear(x, W, b, act=act), z.clamp(min=0) if act == "relu" else z, "out without residual")
    del z
    dy = mk.rows(n, cout, dtype, 2, pad)
    p = mk.mat(n, cout, dtype, 2) if act == "relu" else None
    gx, gw, gb = sc.linear_backward(dy, x, W, p, act=act)
    dz = dy.double() * (p > 0) if act == "relu" else dy.double()
    _same(gx, dz @ W.double().t(), "grad_x")
    _same(gw, x.double().t() @ dz, "grad_W")
    _same(gb, dz.sum(0), "grad_b")


# 20011 x 136 / 328 -> 136: two buffers in both gate kernels, dx on blocked rows with
# three, both weight gradients on 256 x 256 tiles, one with h blocked; 33001 x 64 /
# 512 -> 512: the second product on 256 x 256 tiles; the others odd widths, and few
# tiles.
GATED = [(20011, 136, 328, 136, 0), (33001, 64, 512, 512, 0), (20011, 136, 328, 72, 8), (24001, 100, 267, 131, 3), (1001, 96, 200, 64, 1)]


@gpu
@TYPES
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated_ffn_whole_numbers(dev, shape, act, dtype):
    sc = _sc()
    n, cin, F, cout, pad = shape
    mk = Whole(dev, n + F)
    x = mk.rows(n, cin, dtype, 2, pad)
    Wi, Wo = mk.few(cin, 2 * F, dtype, 4), mk.few(cout, F, dtype, 2).t().contiguous()
    bi, bo, res = mk.vec(2 * F, 2), mk.vec(cout, 9), mk.rows(n, cout, dtype, 9, pad)
    # |g|, |u| <= 4 * 2 + 2, |h| <= 100
    z = x.double() @ Wi.double() + bi.double()
    a = z[:, :F].clamp(min=0) if act == "relu" else z[:, :F]
    ref = (a * z[:, F:]) @ Wo.double() + bo.double() + res.double()
    out, pre = sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res, return_pre=True)
    _same(pre, z, "pre")
    _same(out, ref, "out")
    _same(sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res), ref, "out without pre")
    del z, a, ref
    # |dh| <= 2 * 1 (two entries a row of W_out), |dg|, |du| <= 2 * 8, |h| <= 64
    dy, pre = mk.rows(n, cout, dtype, 1, pad), mk.mat(n, 2 * F, dtype, 8)
    grads = sc.gated_ffn_backward(dy, x, Wi, Wo, pre, act=act)
    g, u, dh = pre[:, :F].double(), pre[:, F:].double(), dy.double() @ Wo.double().t()
    a, d = (g.clamp(min=0), (g > 0).double()) if act == "relu" else (g, torch.ones_like(g))
    dz = torch.cat([dh * u * d, dh * a], 1)
    for got, ref, what in zip(grads, (dz @ Wi.double().t(), x.double().t() @ dz, dz.sum(0),
                                      (a * u).t() @ dy.double(), dy.double().sum(0)),
                              ("grad_x", "grad_W_in", "grad_b_in", "grad_W_out", "grad_b_out")):
        _same(got, ref, what)


# The one-kernel block: 16 rows a wave up to 32768 rows, then 32; kernels of 64
# and of 128 channels, widths below them and unequal, a last workgroup in part.
ONE_KERNEL = [(16385, 65, 65, 128, 3), (20000, 128, 200, 9, 0), (32768, 100, 267, 100, 1), (16384, 120, 33, 127, 0),
              (32769, 65, 65, 128, 0), (40077, 128, 200, 9, 3), (33000, 8, 96, 100, 8), (65536, 100, 512, 128, 0),
              (9, 64, 100, 64, 1), (1000, 40, 33, 17, 0), (32768, 64, 64, 64, 8), (40001, 24, 300, 64, 3)]


@gpu
@TYPES
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("shape", ONE_KERNEL, ids=str)
def test_one_kernel_gated_ffn_whole_numbers(dev, shape, act, dtype):
    sc = _sc()
    n, cin, F, cout, pad = shape
    mk = Whole(dev, n + F + cin)
    x = mk.rows(n, cin, dtype, 2, pad)
    Wi, Wo = mk.few(cin, 2 * F, dtype, 4), mk.mat(F, cout, dtype, 1)
    bi, bo, res = mk.vec(2 * F, 2), mk.vec(cout, 9), mk.rows(n, cout, dtype, 9, pad)
    z = x.double() @ Wi.double() + bi.double()
    a = z[:, :F].clamp(min=0) if act == "relu" else z[:, :F]
    ref = (a * z[:, F:]) @ Wo.double()
    _same(sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res), ref + bo.double() + res.double(), "out")
    z = x.double() @ Wi.double()
    a = z[:, :F].clamp(min=0) if act == "relu" else z[:, :F]
    _same(sc.gated_ffn(x, Wi, None, Wo, None, act=act), (a * z[:, F:]) @ Wo.double(), "out without bias and residual")


@gpu
@TYPES
@pytest.mark.parametrize("act", od.ACTS)
@pytest.mark.parametrize("n", [16384 + 77, 32768 + 77])
@pytest.mark.parametrize("cin,F,cout", [(100, 72, 128), (56, 72, 64)])
def test_one_kernel_gated_ffn_every_activation(dev, n, act, dtype, cin, F, cout):
    """Against the oracle at rows of both ends and of the workgroups' seams.
    Tolerance: fp32 sums of K terms (K + 4) v each, an activation within 32 v (1 +
    |z|) and its slope at most 1.2, one rounding of h and one of out."""
    sc = _sc()
    g = torch.Generator(device=dev).manual_seed(n + cin)

    def normal(*shape, scale=1.0, dt=dtype):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dt)

    x, Wi, Wo = normal(n, cin), normal(cin, 2 * F, scale=cin ** -0.5), normal(F, cout, scale=F ** -0.5)
    bi, bo = normal(2 * F, scale=0.3, dt=torch.float32), normal(cout, scale=0.3, dt=torch.float32)
    res = normal(n, cout)
    out = sc.gated_ffn(x, Wi, bi, Wo, bo, act=act, residual=res)
    at = torch.tensor([0, 1, 15, 16, 31, 32, 63, 64, 127, 128, 8191, 8192, n - 78, n - 77, n - 2, n - 1], device=dev)
    xn, wi, wo, b1, b2, rn = _np(x[at]), _np(Wi), _np(Wo), _np(bi), _np(bo), _np(res[at])
    ro, rz, h = od.gated_ffn(xn, wi, b1, wo, b2, act, rn)
    u, tiny = U[dtype], TINY[dtype]
    ez = (cin + 4) * V * (np.abs(xn) @ np.abs(wi) + np.abs(b1))
    gate, up = rz[:, :F], rz[:, F:]
    a, _ = od.act(gate, act)
    eh = (1.2 * ez[:, :F] + 32 * V * (1 + np.abs(gate))) * (np.abs(up) + ez[:, F:]) + np.abs(a) * ez[:, F:] \
        + (4 * V + u) * np.abs(h) + tiny
    tol = eh @ np.abs(wo) + (F + 4) * V * (np.abs(h) @ np.abs(wo) + np.abs(b2)) + 2 * V * np.abs(rn) \
        + u * np.abs(ro) + tiny
    err = np.abs(_np(out[at]) - ro)
    assert (err <= tol).all(), float(np.nanmax(err / tol))


@gpu
def test_norm_rows_past_32_bits(dev):
    """Norm rows and gradients past element 2^31, with a NaN row after the last,
    at the bounds of the small sizes: fp32 statistics of C values within (C + 8) v of
    the terms summed, one rounding of the result."""
    sc = _sc()
    n, c, half = 17_000_000, 128, torch.float16
    e, u = (c + 8) * V, U[half]
    edge = 2 ** 31 // c
    at = torch.tensor([0, 1, edge - 1, edge, edge + 1, n - 2, n - 1], device=dev)
    g = torch.Generator(device=dev).manual_seed(6)
    buf = torch.empty((n + 1, c), dtype=half, device=dev).normal_(0.5, 1.0, generator=g)
    buf[n] = float("nan")
    x = buf[:n]
    y, mean, rstd = sc.layer_norm(x, return_stats=True)
    xn = _np(x[at])
    ry, rm, rr = od.layer_norm(xn, None, None, 1e-5)
    em = e * np.abs(xn).mean(1)
    sd = np.sqrt(((xn - rm[:, None]) ** 2).mean(1))
    er = rr * (e + (2 * em * sd + em * em) * rr ** 2)
    assert (np.abs(_np(mean[at]) - rm) <= em + V * np.abs(rm)).all()
    assert (np.abs(_np(rstd[at]) - rr) <= er).all()
    a = np.abs(xn - rm[:, None])
    ex = V * (np.abs(xn) + np.abs(rm[:, None]))
    tol = (a + ex) * er[:, None] + rr[:, None] * (em[:, None] + ex) + 4 * V * a * rr[:, None] + u * np.abs(ry) + 2.0 ** -24
    assert (np.abs(_np(y[at]) - ry) <= tol).all()
    gx, gw, gb = sc.layer_norm_backward(y, x, mean, rstd)
    dyn, mn, rn = _np(y[at]), _np(mean[at]), _np(rstd[at])
    rx, _, _ = od.layer_norm_backward(dyn, xn, mn, rn, None)
    xh = (xn - mn[:, None]) * rn[:, None]
    exh = 4 * V * (np.abs(xn) + np.abs(mn[:, None])) * rn[:, None] + 4 * V * np.abs(xh)
    ad = np.abs(dyn)
    s1, s2 = ad.mean(1, keepdims=True), (ad * np.abs(xh)).mean(1, keepdims=True)
    es2 = e * s2 + (ad * exh).mean(1, keepdims=True)
    tol = rn[:, None] * (8 * V * (ad + s1 + np.abs(xh) * s2) + e * s1 + np.abs(xh) * es2 + exh * s2)
    assert (np.abs(_np(gx[at]) - rx) <= tol + u * np.abs(rx) + 2.0 ** -24).all()
    # column sums: 1024 runs of n / 1024 rows, then their sums
    terms = y.double().abs().sum(0)
    assert bool(((gb.double() - y.double().sum(0)).abs() <= (n / 1024 + 2000) * V * terms).all())
    assert bool(gw.isfinite().all())


@gpu
def test_linear_of_more_rows_than_32_bits_count_pieces_of(dev):
    """540 million rows of an odd width: a padded copy of more than 2^30 pieces and
    2^33 elements; rows around element 2^31 and 2^32 of input, copy and result, and
    both ends."""
    sc = _sc()
    n, cin, cout, half = 540_000_000, 9, 8, torch.float16
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((n, cin), dtype=half, device=dev)
    for part in x.split(1 << 26):
        part.copy_(torch.randint(-2, 3, part.shape, generator=g, device=dev, dtype=torch.int8))
    mk = Whole(dev, 4)
    W, b = mk.mat(cin, cout, half, 2), mk.vec(cout, 9)
    out = sc.linear(x, W, b)
    edges = [e // w for e in (2 ** 31, 2 ** 32, 2 ** 33) for w in (9, 16, 8) if e // w < n - 1]
    at = torch.tensor([0, 1, n - 2, n - 1] + [e + d for e in edges for d in (-1, 0, 1)], device=dev)
    _same(out[at], x[at].double() @ W.double() + b.double(), "out")


@gpu
@TYPES
@pytest.mark.parametrize("n,cin,cout", [(5, 33, 77), (8, 64, 8200), (130, 64, 128), (300, 72, 130), (66001, 512, 520),
                                        (33001, 136, 264)])
def test_linear_into_its_residual(dev, n, cin, cout, dtype):
    """The C entry point takes the residual itself as its result, on every kernel."""
    sc = _sc()
    lib = sc.load_library()
    mk = Whole(dev, n)
    x, W, b = mk.mat(n, cin, dtype, 2), mk.mat(cin, cout, dtype, 2), mk.vec(cout, 9)
    res = mk.mat(n, cout, dtype, 9)
    ref = sc.linear(x, W, b, act="relu", residual=res)
    nb = lib.submconv_linear_workspace_bytes(n, cin, cout, 0)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    sc._check(lib.submconv_linear(sc._ptr(x), cin, n, sc._ptr(W), sc._ptr(b), sc._ptr(res), cout, sc._ptr(res), None,
                                  cin, cout, 1, 0 if dtype == torch.float16 else 1, sc._ptr(ws), nb, sc._stream(dev)))
    assert torch.equal(res, ref)


@gpu
@pytest.mark.parametrize("n,cin,F,cout", [(20001, 64, 256, 64), (20001, 128, 512, 128), (40001, 100, 267, 72),
                                          (300, 72, 136, 200), (5, 16, 40, 16)])
def test_gated_ffn_within_its_workspace(dev, n, cin, F, cout):
    """The call without pre runs in exactly what its query gives and writes nothing
    past it."""
    sc = _sc()
    lib = sc.load_library()
    half = torch.float16
    mk = Whole(dev, n)
    x, Wi, Wo = mk.mat(n, cin, half, 2), mk.few(cin, 2 * F, half, 4), mk.mat(F, cout, half, 1)
    aligned = int(cin % 8 == 0 and F % 8 == 0 and cout % 8 == 0)
    nb = lib.submconv_gated_ffn_inference_workspace_bytes(n, cin, F, cout, aligned)
    ws = torch.full((nb + 256,), 9, dtype=torch.uint8, device=dev)
    out = torch.full((n + 1, cout), 7.0, dtype=half, device=dev)

    def call(nbytes):
        return lib.submconv_gated_ffn(sc._ptr(x), cin, n, sc._ptr(Wi), None, sc._ptr(Wo), None, None, 0, sc._ptr(out),
                                      None, cin, F, cout, 1, 0, sc._ptr(ws), nbytes, sc._stream(dev))

    if nb and aligned:  # (for unaligned sizes the query counts a copy of every operand)
        assert call(nb - 1) == -1
    sc._check(call(nb))
    z = x.double() @ Wi.double()
    _same(out[:n], (z[:, :F].clamp(min=0) * z[:, F:]) @ Wo.double(), "out")
    assert bool((out[n] == 7).all()) and bool((ws[nb:] == 9).all())


@gpu
@TYPES
@pytest.mark.parametrize("n", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("cin,cout", [(1027, 257), (1028, 257), (4099, 1024), (4095, 1024), (4100, 1025), (8191, 300)])
def test_linear_few_rows_of_a_long_k(dev, n, cin, cout, dtype):
    """Either side of the rule that gives long walks along k narrow strips."""
    sc = _sc()
    mk = Whole(dev, n * cin)
    x, W, b, res = mk.rows(n, cin, dtype, 2, 3), mk.mat(cin, cout, dtype, 2), mk.vec(cout, 9), mk.rows(n, cout, dtype, 9, 3)
    out, pre = sc.linear(x, W, b, act="relu", residual=res, return_pre=True)
    z = x.double() @ W.double() + b.double()
    _same(pre, z, "pre")
    _same(out, z.clamp(min=0) + res.double(), "out")
