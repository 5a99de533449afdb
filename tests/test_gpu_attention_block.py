"""The attention block on packed items: the operators together, as a model runs
them, against the same block in fp64 torch on the CPU, and its example.

Bound of a whole pass: every stored tensor is off by at most u = 2^-11 (fp16) of
itself, a pass stores 16 of them on its longest way (norm, projections, turned
rows, weights, sums, hidden rows, for both attentions and the feed-forward
block) and its gradient as many again, and a layer of this block enlarges a
relative error at most four times: 16 * 4 * u for the output, twice that for
gradients, in the norm of each tensor."""
import os
import sys

import pytest
import torch

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = 16 * 4 * 2.0 ** -11


def _sc():
    import submanifold_sparse_convolution_hash_amd as sc
    sc.load_library()
    return sc


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _turn(x, at, freqs):
    """Interleaved pairs of the first columns, by the axes one after the other."""
    t = (at.double()[:, :, None] * freqs).flatten(1)[:, None]
    p = t.shape[2]
    a, b = x[..., 0:2 * p:2], x[..., 1:2 * p:2]
    turned = torch.stack([a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * p:]], -1)


def _attend(m, par, name, x, off, at, ctx, coff):
    h, hk, d = m.heads, m.kv_heads, m.dim
    rows = (x @ par[name + "proj_in.weight"] + par[name + "proj_in.bias"]).view(len(x), -1, d)
    if m.own:
        q, k, v, coff = rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:], off
        q, k = _turn(q, at, m.freqs.cpu()), _turn(k, at, m.freqs.cpu())
    else:
        q = rows
        both = (ctx @ par[name + "proj_context.weight"] + par[name + "proj_context.bias"]).view(len(ctx), -1, d)
        k, v = both[:, :hk], both[:, hk:]
    out = []
    for (s, e), (ks, ke) in zip(zip(off, off[1:]), zip(coff, coff[1:])):
        kk, vv = (t[ks:ke].repeat_interleave(h // hk, 1).transpose(0, 1) for t in (k, v))
        z = q[s:e].transpose(0, 1) @ kk.transpose(1, 2) * d ** -0.5
        out.append((torch.softmax(z, 2) @ vv).transpose(0, 1).reshape(e - s, h * d))
    return torch.cat(out) @ par[name + "proj_out.weight"] + par[name + "proj_out.bias"]


def _block(m, par, x, off, at, ctx, coff):
    """The block in fp64, from its formulas."""
    def layer_norm(t, name):
        return torch.nn.functional.layer_norm(t, t.shape[1:], par[name + ".weight"], par[name + ".bias"], 1e-5)

    g = torch.cat([torch.nn.functional.group_norm(x[s:e].T[None], m.norm.groups, par["norm.weight"], par["norm.bias"],
                                                  1e-5)[0].T for s, e in zip(off, off[1:])])
    h = x + _attend(m.attention, par, "attention.", g, off, at, None, None)
    if m.over_context is not None:
        h = h + _attend(m.over_context, par, "over_context.", layer_norm(h, "norm_context"), off, at, ctx, coff)
    z = layer_norm(h, "norm_ffn") @ par["ffn.w_in"] + par["ffn.b_in"]
    gate, up = z.chunk(2, 1)
    return h + (torch.nn.functional.silu(gate) * up) @ par["ffn.w_out"] + par["ffn.b_out"]


@gpu
@pytest.mark.parametrize("lengths", [[130], [40, 1, 300], [700, 900]])
@pytest.mark.parametrize("with_context", [False, True])
def test_block_and_its_gradients(dev, lengths, with_context):
    sc = _sc()
    torch.manual_seed(3)
    c, width = 64, 24
    m = sc.SparseAttentionBlock(c, 96, heads=4, kv_heads=2, groups=8, context=width if with_context else None, rotary=12,
                                device=dev)
    assert m.attention.freqs.dtype == torch.float64
    for p in m.parameters():  # parameters of no special value
        p.data += 0.1 * torch.randn_like(p)
    off = [0] + torch.tensor(lengths).cumsum(0).tolist()
    coff = [5 * i for i in range(len(off))]
    n = off[-1]
    offsets, coffsets = (torch.tensor(t, dtype=torch.int32, device=dev) for t in (off, coff))
    b = torch.arange(len(lengths)).repeat_interleave(torch.tensor(lengths))
    coords = torch.cat([b[:, None], torch.randint(0, 64, (n, 3))], 1).to(torch.int32).to(dev)
    assert sc.item_offsets(coords, len(lengths)).tolist() == off
    x = torch.randn(n, c, device=dev).half().requires_grad_()
    ctx = torch.randn(coff[-1], width, device=dev).half().requires_grad_() if with_context else None
    extra = (ctx, coffsets) if with_context else ()
    y = m(x, offsets, coords[:, 1:], *extra)
    g = torch.randn(n, c, device=dev).half()
    y.backward(g)

    par = {k: v.detach().cpu().double().requires_grad_() for k, v in m.named_parameters()}
    rx = x.detach().cpu().double().requires_grad_()
    rc = ctx.detach().cpu().double().requires_grad_() if with_context else None
    ry = _block(m, par, rx, off, coords[:, 1:].cpu(), rc, coff)
    ry.backward(g.cpu().double())

    def off_by(got, ref):
        return ((got.detach().cpu().double() - ref).norm() / ref.norm()).item()

    assert off_by(y, ry.detach()) <= BOUND
    assert off_by(x.grad, rx.grad) <= 2 * BOUND
    if with_context:
        assert off_by(ctx.grad, rc.grad) <= 2 * BOUND
    for k, v in m.named_parameters():
        assert off_by(v.grad, par[k].grad) <= 2 * BOUND, k
    # without gradients: the same values of the attention, whose queries and keys are
    # then turned in place (the gated block has other kernels there)
    a = m.attention(x, offsets, coords[:, 1:]).detach()
    with torch.no_grad():
        assert off_by(m(x, offsets, coords[:, 1:], *extra), ry.detach()) <= BOUND
        assert torch.equal(m.attention(x, offsets, coords[:, 1:]), a)
    m.requires_grad_(False)
    assert torch.equal(m.attention(x.detach(), offsets, coords[:, 1:]), a)


@gpu
def test_one_item_needs_no_offsets(dev):
    sc = _sc()
    torch.manual_seed(4)
    m = sc.SparseAttentionBlock(32, 32, heads=2, groups=4, context=16, rotary=6, device=dev)
    n = 77
    x, at = torch.randn(n, 32, device=dev).half(), torch.randint(0, 9, (n, 3), device=dev, dtype=torch.int32)
    ctx = torch.randn(5, 16, device=dev).half()
    off, coff = (torch.tensor([0, k], dtype=torch.int32, device=dev) for k in (n, 5))
    assert torch.equal(m(x, None, at, ctx), m(x, off, at, ctx, coff))
    with pytest.raises(ValueError, match="context_offsets"):
        m(x, off, at, ctx)
    with pytest.raises(ValueError, match="positions"):
        m(x, off, None, ctx, coff)
    with pytest.raises(ValueError, match="context"):
        m(x, off, at)


@gpu
def test_module_keeps_its_frequencies(dev):
    """In 64 bits through a change of type, and on the module's device."""
    sc = _sc()
    m = sc.SparseAttention(64, 2, rotary=12)
    m = m.to(torch.bfloat16).to(dev)
    assert m.freqs.dtype == torch.float64 and m.freqs.device == dev
    assert torch.equal(m.freqs.cpu(), sc.rotary_frequencies(12, 3))
    m.proj_in.bias.data, m.proj_out.bias.data = m.proj_in.bias.data.float(), m.proj_out.bias.data.float()
    x = torch.randn(20, 64, device=dev).bfloat16()
    at = torch.randint(0, 9, (20, 3), device=dev, dtype=torch.int32)
    assert torch.isfinite(m(x, positions=at).float()).all()


@gpu
def test_example_trains(dev):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_attention
    finally:
        sys.path.pop(0)
    losses, final = train_attention.train(grid=12, channels=32, steps=3)
    assert len(losses) == 3 and all(v == v and v < 1e6 for v in losses + [final])
