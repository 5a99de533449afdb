"""Sizes whose launches would pass 32 bits of threads, without a GPU."""
import pytest

P = 4096  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    import submanifold_sparse_convolution_hash_amd as sc
    return sc.load_library()


def _heads(rows, heads, dim):
    return (P, heads * dim, dim)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("nq,nk,heads,kv_heads", [(2 ** 27, 2 ** 27, 16, 16), (2 ** 27, 100, 64, 16),
                                                  (2 ** 30, 2 ** 30, 2, 2)])
def test_attention_refuses_more_threads_than_a_launch_has(lib, back, nq, nk, heads, kv_heads):
    q, kv = _heads(nq, heads, 8), _heads(nk, kv_heads, 8)
    args = (*q, nq, *kv, *kv, nk, heads, kv_heads, 8, P, P, None, 1, 0.3, 0)
    if back:
        status = lib.submconv_attention_backward(P, heads * 8, 8, P, P, *args, P, P, P, 0, P, 1 << 50, None)
    else:
        status = lib.submconv_attention(*args, P, P, 0, P, 1 << 50, None)
    assert status == -4 and b"too many" in lib.submconv_last_error()
