"""The attention modules' own checks, without a GPU."""
import pytest
import torch


def _sc():
    import submanifold_sparse_convolution_hash_amd as sc
    return sc


@pytest.mark.parametrize("axes,shape", [(3, (5, 4)), (3, (5, 2)), (3, (5, 1)), (3, (5,)), (1, (5, 2)), (2, (5, 3)),
                                        (1, (5, 1, 1)), (1, ())])
def test_positions_have_the_modules_axes(axes, shape):
    """A batch index among them, or an axis too few, would turn other columns."""
    m = _sc().SparseAttention(64, 1, rotary=12, axes=axes)
    x = torch.zeros((5, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="axes"):
        m(x, positions=torch.zeros(shape, dtype=torch.int32))
    with pytest.raises(TypeError, match="positions"):
        m(x, positions=[1, 2, 3])


@pytest.mark.parametrize("what", [dict(context=torch.zeros((2, 8), dtype=torch.float16)),
                                  dict(context_offsets=torch.zeros(2, dtype=torch.int32))])
def test_a_context_that_nothing_would_read_is_refused(what):
    sc = _sc()
    x = torch.zeros((5, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="context"):
        sc.SparseAttention(64, 2)(x, **what)
    with pytest.raises(ValueError, match="context"):
        sc.SparseAttentionBlock(64, 32, heads=2, groups=8)(x, **what)


def test_made_without_memory_and_given_some_later():
    """On the meta device first: the frequencies are there after to_empty, in 64 bits,
    whatever types the module went through."""
    sc = _sc()
    want = sc.rotary_frequencies(12, 3)
    m = sc.SparseAttention(64, 2, rotary=12, device="meta")
    assert m.freqs.is_meta and m.freqs.dtype == torch.float64
    m = m.to(torch.bfloat16)
    assert m.freqs.is_meta and m.freqs.dtype == torch.float64
    m = m.to_empty(device="cpu")
    assert m.proj_in.weight.device.type == "cpu" and m.proj_in.weight.dtype == torch.bfloat16
    assert m.freqs.dtype == torch.float64 and torch.equal(m.freqs, want)
    m = m.to_empty(device="cpu")  # frequencies that are there stay
    assert torch.equal(m.freqs, want)
    with torch.device("meta"):
        block = sc.SparseAttentionBlock(64, 96, heads=4, groups=8, context=24, rotary=6, axes=1)
    block = block.to_empty(device="cpu")
    assert torch.equal(block.attention.freqs, sc.rotary_frequencies(6, 1)) and block.over_context.freqs is None


@pytest.mark.parametrize("kw", [dict(heads=0), dict(heads=-4), dict(heads=0, dim=16), dict(heads=4, kv_heads=0)])
def test_no_heads_are_refused(kw):
    with pytest.raises(ValueError):
        _sc().SparseAttention(64, **kw)
