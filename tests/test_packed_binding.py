"""Host side of the operators on packed items, without a GPU: what the entry
points refuse before anything is enqueued, workspaces, modules."""
import ctypes

import pytest
import torch

P = 4096  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    import submanifold_sparse_convolution_hash_amd as sc
    return sc.load_library()


def _message(lib):
    return lib.submconv_last_error().decode()


def _group(lib, back=False, **kw):
    a = dict(x=P, ldx=32, n=10, c=32, g=4, off=P, items=2, eps=1e-5, act=0, y=P, dtype=0, ws=P, nb=1 << 30)
    a.update(kw)
    if back:
        return lib.submconv_group_norm_backward(a["y"], a["ldx"], a["x"], a["ldx"], a["n"], a["c"], a["g"], a["off"],
                                                a["items"], kw.get("mean", P), P, None, None, a["act"], P, P, P,
                                                a["dtype"], a["ws"], a["nb"], None)
    return lib.submconv_group_norm(a["x"], a["ldx"], a["n"], a["c"], a["g"], a["off"], a["items"], None, None, a["eps"],
                                   a["act"], a["y"], None, None, a["dtype"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(n=2 ** 31), -1), (dict(c=0), -4), (dict(c=8193, ldx=9000), -4), (dict(g=0), -1),
    (dict(g=5), -1), (dict(items=0), -1), (dict(items=65536), -1), (dict(off=None), -1), (dict(act=9), -1),
    (dict(dtype=3), -1), (dict(x=None), -1), (dict(x=P + 1), -1), (dict(dtype=2, x=P + 2), -1), (dict(ldx=31), -1),
    (dict(y=None), -1), (dict(n=5000, nb=0), -1), (dict(n=5000, ws=None), -1), (dict(n=5000, ws=P + 4), -1)])
def test_group_norm_refuses(lib, kw, status, back):
    assert _group(lib, back, **kw) == status and _message(lib)


def test_group_norm_refuses_more(lib):
    assert _group(lib, eps=-1.0) == -1 and _group(lib, eps=float("nan")) == -1
    assert _group(lib, True, mean=None) == -1
    q = lib.submconv_group_norm_workspace_bytes
    assert q(64, 256, 32, 2, 0) == 0 and q(209715, 128, 32, 1, 0) > 0 and q(10, 30, 4, 1, 0) == -1
    assert lib.submconv_group_norm_backward_workspace_bytes(10, 0, 4, 1, 0) == -4


def _turn(lib, **kw):
    a = dict(x=P, ldx=64, hx=32, n=10, h=2, d=32, pos=P, axes=1, f=P, nf=16, out=2 * P, ldo=64, ho=32, dtype=0)
    a.update(kw)
    return lib.submconv_rotary(a["x"], a["ldx"], a["hx"], a["n"], a["h"], a["d"], a["pos"], 1, 1, a["axes"], a["f"],
                               a["nf"], 0, 0, 1.0, a["out"], a["ldo"], a["ho"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), -1), (dict(h=0), -4), (dict(d=1), -4), (dict(axes=0), -4), (dict(axes=5), -4), (dict(nf=0), -1),
    (dict(nf=17), -1), (dict(axes=2, nf=9), -1), (dict(nf=2 ** 30, axes=4), -1), (dict(dtype=7), -1),
    (dict(x=None), -1), (dict(out=None), -1), (dict(hx=31), -1), (dict(ldx=63), -1), (dict(ldo=10), -1),
    (dict(pos=None), -1), (dict(f=None), -1), (dict(f=P + 4), -1), (dict(pos=P + 2), -1), (dict(x=P + 1), -1),
    (dict(out=P, ldo=80), -1)])
def test_rotary_refuses(lib, kw, status):
    assert _turn(lib, **kw) == status and _message(lib)


def test_nothing_to_do_is_fine(lib):
    assert _turn(lib, n=0, x=None, out=None, pos=None, f=P) == 0
    assert _group(lib, n=0, x=None, y=None) == 0
    assert _attn(lib, nq=0, q=None, out=None) == 0
    assert lib.submconv_item_offsets(None, 4, -1, 1, P, P, None) == -1
    assert lib.submconv_item_offsets(P, 4, 5, 0, P, P, None) == -1
    assert lib.submconv_item_offsets(None, 4, 5, 1, P, P, None) == -1
    assert lib.submconv_item_offsets(P, 4, 5, 1, P, None, None) == -1


def _attn(lib, back=False, **kw):
    a = dict(q=P, ldq=128, hq=32, nq=10, k=P, ldk=64, hk=32, v=P, nk=20, h=4, kvh=2, d=32, off=P, koff=P, items=2,
             scale=0.2, out=P, lse=P, dtype=0, ws=P, nb=1 << 30, grad=P)
    a.update(kw)
    args = (a["q"], a["ldq"], a["hq"], a["nq"], a["k"], a["ldk"], a["hk"], a["v"], a["ldk"], a["hk"], a["nk"], a["h"],
            a["kvh"], a["d"], a["off"], a["koff"], None, a["items"], a["scale"], 0)
    if back:
        return lib.submconv_attention_backward(P, a["ldq"], a["hq"], a["out"], a["lse"], *args, a["grad"], P, P,
                                               a["dtype"], a["ws"], a["nb"], None)
    return lib.submconv_attention(*args, a["out"], a["lse"], a["dtype"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -1), (dict(nq=-1), -1), (dict(nk=2 ** 31), -1), (dict(kvh=0), -1), (dict(h=3), -1),
    (dict(h=0, kvh=1), -1), (dict(d=0), -4), (dict(d=136, ldq=544, hq=136, ldk=272, hk=136), -4), (dict(d=20), -4),
    (dict(items=0), -1), (dict(items=65536), -1), (dict(off=None), -1), (dict(koff=None), -1), (dict(scale=0.0), -1),
    (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(q=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(q=P + 2), -1), (dict(k=P + 8), -1), (dict(ldq=132), -1),
    (dict(hq=36), -1), (dict(ldk=60), -1), (dict(hk=24), -1), (dict(ldk=2 ** 22 + 8), -4), (dict(out=None), -1),
    (dict(out=P + 4), -1)])
def test_attention_refuses(lib, kw, status, back):
    assert _attn(lib, back, **kw) == status and _message(lib)


def test_attention_refuses_more(lib):
    assert _attn(lib, True, lse=None) == -1 and _attn(lib, True, grad=P + 2) == -1
    assert _attn(lib, True, nb=0) == -1 and _attn(lib, True, ws=None) == -1
    assert _attn(lib, nk=100000, nb=0) == -1  # the keys are split: a workspace is needed
    q = lib.submconv_attention_workspace_bytes
    assert q(20000, 20000, 12, 12, 64, 1, 0) == 0 and q(1, 30000, 16, 4, 64, 1, 1) > 0
    assert q(10, 10, 3, 2, 64, 1, 0) == -1 and q(10, 10, 2, 2, 60, 1, 0) == -4
    assert lib.submconv_attention_backward_workspace_bytes(10, 10, 2, 0, 64, 1, 0) == -1


def test_host_tensors_are_refused():
    import submanifold_sparse_convolution_hash_amd as sc

    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        sc.group_norm(x, 2)
    with pytest.raises(ValueError, match="device tensor"):
        sc.rotary(x.view(4, 1, 8), torch.zeros(4, dtype=torch.int32), sc.rotary_frequencies(8))
    with pytest.raises(ValueError, match="device tensor"):
        sc.attention(*[x.half().view(4, 1, 8)] * 3)
    with pytest.raises(ValueError, match="device tensor"):
        sc.item_offsets(torch.zeros((2, 4), dtype=torch.int32))
    with pytest.raises(TypeError, match="must be a tensor"):
        sc.attention(None, None, None)


@pytest.mark.parametrize("kw", [dict(dim=7), dict(dim=8, axes=3), dict(dim=0), dict(dim=8, base=0.0),
                                dict(dim=8, factor=-1.0), dict(dim=8, scaling="other"),
                                dict(dim=8, scaling="parts", low=4, high=4), dict(dim=8, axes=0)])
def test_rotary_frequencies_refuses(kw):
    import submanifold_sparse_convolution_hash_amd as sc

    with pytest.raises(ValueError):
        sc.rotary_frequencies(**kw)


def test_group_norm_module_records_only_where_something_requires_a_gradient(monkeypatch):
    from submanifold_sparse_convolution_hash_amd import packed

    monkeypatch.setattr(packed, "group_norm", lambda *a: "plain")
    monkeypatch.setattr(packed.GroupNormFunction, "apply", lambda *a: "recorded")
    m, x = packed.GroupNorm(2, 8, act="silu"), torch.zeros(2, 8)
    assert m(x) == "recorded"
    m.requires_grad_(False)
    assert m(x) == "plain" and m(x.requires_grad_()) == "recorded"
    with pytest.raises(ValueError):
        packed.GroupNorm(3, 8)
    with pytest.raises(ValueError):
        packed.GroupNorm(2, 8, act="other")


@pytest.mark.parametrize("kw", [dict(heads=3), dict(heads=4, kv_heads=3), dict(heads=0), dict(heads=16, dim=4),
                                dict(heads=2, dim=136), dict(heads=4, dim=20), dict(heads=4, rotary=18),
                                dict(heads=4, rotary=10), dict(heads=4, rotary=12, context=8)])
def test_attention_module_refuses(kw):
    import submanifold_sparse_convolution_hash_amd as sc

    with pytest.raises((ValueError, ZeroDivisionError)):
        sc.SparseAttention(64, **kw)
