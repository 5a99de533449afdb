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
