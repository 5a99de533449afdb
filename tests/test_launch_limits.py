"""Sizes whose launches would pass 32 bits of threads are refused before anything
is enqueued: a launch cuts the count without an error. Without a GPU."""
import ctypes

import pytest

P = 4096  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    import submanifold_sparse_convolution_hash_amd as sc
    return sc.load_library()


def _refused(lib, status):
    return status == -4 and b"too many" in lib.submconv_last_error()


@pytest.mark.parametrize("n,flags", [(2 ** 28, 0x2), (2 ** 29, 0)])
def test_map_build(lib, n, flags):
    """A thread per row and tap: 27 with sorted keys, 14 with the table."""
    import submanifold_sparse_convolution_hash_amd as sc

    assert sc.FLAG_SORTED_KEYS == 0x2
    grid, out = (ctypes.c_int32 * 3)(4096, 4096, 4096), ctypes.c_void_p()
    assert _refused(lib, lib.submconv_build_map(P, n, 1, grid, flags, None, ctypes.byref(out)))
    assert not out.value


@pytest.mark.parametrize("n,c", [(2 ** 26, 64), (2 ** 29, None), (2 ** 40, None)])
def test_subdivide(lib, n, c):
    feats = None if c is None else P
    assert _refused(lib, lib.submconv_subdivide(P, n, feats, c or 0, P, feats, None))


def test_linear(lib):
    n, cin, cout = 2 ** 32, 8, 8
    args = (P, cin, n, P, None, None, 0, P, None, cin, cout, 0, 0)
    assert _refused(lib, lib.submconv_linear(*args, P, 1 << 50, None))


def test_gated_block(lib):
    n, c, hidden = 2 ** 32, 8, 16
    for pre in (None, P):  # hidden rows in registers, and in memory
        args = (P, c, n, P, None, P, None, None, 0, P, pre, c, hidden, c, 2, 0)
        assert _refused(lib, lib.submconv_gated_ffn(*args, P, 1 << 50, None))
