"""Calls on packed items that are out of the ordinary: batches without rows,
gradients that start anywhere, batch indices without end, the largest sizes."""
import pytest
import torch

gpu = pytest.mark.gpu


def _sc():
    import submanifold_sparse_convolution_hash_amd as sc
    sc.load_library()
    return sc


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _randn(shape, dtype, dev, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev)


@gpu
def test_rotary_of_more_rows_than_a_launch_has_workgroups(dev):
    """2^24 workgroups of 256 threads pass a launch's 32 bits: with so many rows a
    workgroup takes more than one, however wide they are. 17 GB, in place."""
    sc = _sc()
    n, d = 2 ** 24 + 5, 514
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.zeros((n, 1, d), dtype=torch.bfloat16, device=dev)
    f = sc.rotary_frequencies(d, device=dev)
    at = torch.arange(n, dtype=torch.int32, device=dev)
    for interleaved in (False, True):
        pieces = [slice(0, 5), slice(2 ** 23 - 3, 2 ** 23 + 4), slice(n - 9, n)]
        want = []
        for i, p in enumerate(pieces):
            x[p] = _randn((p.stop - p.start, 1, d), torch.bfloat16, dev, i)
            want.append(sc.rotary(x[p].clone(), at[p], f, interleaved))
        assert sc.rotary(x, at, f, interleaved, out=x) is x
        for p, w in zip(pieces, want):
            assert torch.equal(x[p], w), p
            x[p] = 0.0
        assert not x.any()  # the rows between them, which were zeros


@gpu
@pytest.mark.parametrize("items", [None, 1, 3])
@pytest.mark.parametrize("context_rows", [None, 0, 7])
def test_block_without_rows(dev, items, context_rows):
    """No sites: an output of no rows, gradients of zero."""
    sc = _sc()
    width = None if context_rows is None else 24
    m = sc.SparseAttentionBlock(64, 96, heads=4, kv_heads=2, groups=8, context=width, rotary=12, device=dev)
    x = torch.zeros((0, 64), dtype=torch.float16, device=dev, requires_grad=True)
    at = torch.zeros((0, 3), dtype=torch.int32, device=dev)
    off = None if items is None else torch.zeros(items + 1, dtype=torch.int32, device=dev)
    extra = ()
    if context_rows is not None:
        ctx = _randn((context_rows, width), torch.float16, dev, 1).requires_grad_()
        coff = None if items is None else torch.tensor([0] * items + [context_rows], dtype=torch.int32, device=dev)
        extra = (ctx, coff)
    with torch.no_grad():
        assert m(x, off, at, *extra).shape == (0, 64)
    y = m(x, off, at, *extra)
    assert y.shape == (0, 64) and y.requires_grad
    y.backward(torch.zeros_like(y))
    assert x.grad.shape == (0, 64)
    for name, p in m.named_parameters():
        assert p.grad is not None and p.grad.shape == p.shape and not p.grad.any(), name
    if context_rows is not None:
        assert ctx.grad.shape == ctx.shape and not ctx.grad.any()


@gpu
def test_attention_over_a_context_without_rows(dev):
    """Sites that attend to nothing get the last product's bias."""
    sc = _sc()
    m = sc.SparseAttention(32, 2, context=16, device=dev)
    m.proj_out.bias.data += torch.linspace(-1, 1, 32, device=dev)
    x = _randn((9, 32), torch.float16, dev, 2).requires_grad_()
    ctx = torch.zeros((0, 16), dtype=torch.float16, device=dev, requires_grad=True)
    y = m(x, context=ctx)
    assert torch.equal(y, m.proj_out.bias.data.half().expand(9, 32))
    y.backward(torch.ones_like(y))
    assert not x.grad.any() and ctx.grad.shape == (0, 16)
    assert not m.proj_in.weight.grad.any() and not m.proj_context.weight.grad.any()


@gpu
@pytest.mark.parametrize("start", [1, 3, 8])
def test_attention_gradient_that_starts_anywhere(dev, start):
    """The gradient of a tensor that was joined with others is a piece of theirs."""
    sc = _sc()
    q, k, v = (_randn((50, h, 40), torch.float16, dev, h).requires_grad_() for h in (4, 2, 2))
    other = torch.zeros(start, dtype=torch.float16, device=dev, requires_grad=True)
    out = sc.AttentionFunction.apply(q, k, v, None, None, None, True, None)
    g = _randn((start + out.numel(),), torch.float16, dev, 7)
    torch.cat([other, out.flatten()]).backward(g)
    with torch.no_grad():
        o, lse = sc.attention(q, k, v, causal=True, return_lse=True)
        want = sc.attention_backward(g[start:].clone().view_as(o), q, k, v, o, lse, causal=True)
    assert torch.equal(o, out)
    for t, w in zip((q, k, v), want):
        assert torch.equal(t.grad, w)


@gpu
@pytest.mark.parametrize("index", [65535, 2 ** 31 - 2, 2 ** 31 - 1])
def test_item_offsets_allocates_nothing_for_an_index_past_every_batch(dev, index):
    sc = _sc()
    coords = torch.zeros((600, 4), dtype=torch.int32, device=dev)
    coords[599, 0] = index
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(sc.SubmconvError, match="items"):
        sc.item_offsets(coords)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


@gpu
def test_rotary_in_place_is_seen_by_autograd(dev):
    """A tensor that a recorded operation keeps for its gradient is turned in place:
    the backward pass refuses it, as after any change in place."""
    sc = _sc()
    at, f = torch.arange(9, dtype=torch.int32, device=dev), sc.rotary_frequencies(32, device=dev)
    x = _randn((9, 2, 32), torch.float32, dev, 1)
    w = torch.ones_like(x, requires_grad=True)
    y = (x * w).sum()
    sc.rotary(x, at, f)  # elsewhere: x is as it was
    y.backward(retain_graph=True)
    sc.rotary(x, at, f, out=x)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():  # tensors without a version
        z = x.clone()
        assert sc.rotary(z, at, f, out=z) is z


@gpu
@pytest.mark.parametrize("rows", [3, 40])
def test_most_items(dev, rows):
    """65535 items, as many as there may be, of one length, the last of them without
    rows: the same as a batch of matrices in fp64."""
    sc = _sc()
    items, h, d = 65535, 2, 16
    n = (items - 1) * rows
    off = (torch.arange(items + 1, device=dev).clamp(max=items - 1) * rows).to(torch.int32)
    x = _randn((n, h * d), torch.float32, dev, rows)
    w, b = (_randn((h * d,), torch.float32, dev, s) for s in (1, 2))
    y, mean, rstd = sc.group_norm(x, 4, w, b, offsets=off, return_stats=True)
    t = x.double().view(items - 1, rows, 4, -1)
    m, v = t.mean((1, 3), keepdim=True), t.var((1, 3), keepdim=True, correction=0)
    xh = (t - m) * (v + 1e-5).rsqrt()
    # a few roundings of values below 8, and of a deviation that may be small
    e = 2.0 ** -24 * 64 * (1 + (v + 1e-5).rsqrt())
    bound = (e * 8 * w.abs().double().view(4, -1) + 2.0 ** -20 * (1 + b.abs().double().view(4, -1))).expand_as(t)
    assert ((y.double().view_as(t) - (xh * w.double().view(4, -1) + b.double().view(4, -1))).abs() <= bound).all()
    assert mean[-1].eq(0).all() and (mean[:-1].double() - m[:, 0, :, 0]).abs().max().item() <= 2.0 ** -24 * 64 * 8
    g = _randn((n, h * d), torch.float32, dev, 5)
    _, gw, gb = sc.group_norm_backward(g, x, mean, rstd, w, b, offsets=off)
    gd = g.double()
    terms = gd * xh.flatten(2).reshape(n, -1)
    # sums in parts: some hundreds of steps, 2^-24 of the sum of sizes each
    assert ((gb.double() - gd.sum(0)).abs() <= 2.0 ** -24 * 2000 * gd.abs().sum(0)).all()
    assert ((gw.double() - terms.sum(0)).abs() <= 2.0 ** -24 * 2000 * (gd.abs() * 8).sum(0)).all()
    q = x.half().view(n, h, d)
    out, lse = sc.attention(q, q, q, off, causal=True, return_lse=True)
    p = q.double().view(items - 1, rows, h, d).transpose(1, 2)
    s = p @ p.transpose(2, 3).contiguous() * d ** -0.5
    s = s.masked_fill(torch.ones((rows, rows), dtype=torch.bool, device=dev).triu(1), float("-inf"))
    want = torch.softmax(s, 3) @ p
    size = torch.softmax(s, 3) @ p.abs()
    err = (out.double().view(items - 1, rows, h, d).transpose(1, 2) - want).abs()
    # a weight's rounding, its score's and the sums', the stored value's
    assert (err <= 2.0 ** -11 * size + 2.0 ** -15 * size + 2.0 ** -11 * want.abs() + 2.0 ** -24).all()
    assert (lse.double().view(items - 1, rows, h).transpose(1, 2) - s.logsumexp(3)).abs().max().item() <= 2.0 ** -16
