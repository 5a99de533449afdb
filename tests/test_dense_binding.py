"""Host side of the dense layers' binding, without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_package_imports_on_a_torch_without_gpu_support():
    """Only a torch built for GPUs has the private raw-stream call."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import submanifold_sparse_convolution_hash_amd as sc\n"
            "assert callable(sc.linear)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("kind", ["LayerNorm", "Linear", "GatedFeedForward"])
def test_modules_record_only_where_something_requires_a_gradient(kind, monkeypatch):
    """A frozen module keeps nothing for a backward pass that cannot come (the
    gated block would write its pre-activations and take slower kernels)."""
    from submanifold_sparse_convolution_hash_amd import dense

    name = {"LayerNorm": "layer_norm", "Linear": "linear", "GatedFeedForward": "gated_ffn"}[kind]
    monkeypatch.setattr(dense, name, lambda *a: "plain")
    monkeypatch.setattr(getattr(dense, kind + "Function"), "apply", lambda *a: "recorded")
    sizes = {"LayerNorm": (8,), "Linear": (8, 4), "GatedFeedForward": (8, 4)}[kind]
    m = getattr(dense, kind)(*sizes)
    x = torch.zeros(2, 8, dtype=torch.float16)
    assert m(x) == "recorded"
    with torch.no_grad():
        assert m(x) == "plain"
    m.requires_grad_(False)
    assert m(x) == "plain"
    for p in m.parameters():  # any one of them is enough
        p.requires_grad_(True)
        assert m(x) == "recorded"
        p.requires_grad_(False)
    y = x.clone().requires_grad_()
    assert m(y) == "recorded"
    if kind != "LayerNorm":
        assert m(x, x) == "plain" and m(x, y) == "recorded"


def test_workspace_of_the_gated_block():
    """Where the hidden rows stay in registers no workspace is asked for them;
    the query for calls with pre covers both."""
    import submanifold_sparse_convolution_hash_amd as sc

    lib = sc.load_library()
    keep, alone = lib.submconv_gated_ffn_workspace_bytes, lib.submconv_gated_ffn_inference_workspace_bytes
    assert keep(209715, 128, 512, 128, 1) >= 209715 * 512 * 2
    assert alone(209715, 128, 512, 128, 1) == 0
    assert alone(20000, 64, 256, 64, 1) == 0
    # odd widths still go through padded copies, of x (104 columns) among others
    assert 209715 * 104 * 2 <= alone(209715, 100, 267, 100, 0) < 209715 * 112 * 2
    for n in (0, 1, 8, 9, 1000, 20000, 100000):
        for cin, hidden, cout in ((64, 256, 64), (128, 512, 128), (129, 512, 128), (256, 1024, 256), (33, 2049, 20)):
            for aligned in (0, 1):
                a, k = alone(n, cin, hidden, cout, aligned), keep(n, cin, hidden, cout, aligned)
                assert 0 <= a <= k
                if max(cin, cout) > 128 or hidden > 2048:
                    assert a == k
    assert alone(-1, 8, 16, 8, 0) == -1 and alone(9, 8, 0, 8, 0) == -4


def test_one_kernel_or_two_by_the_length_of_the_walk():
    """One workgroup walks all hidden channels in the one-kernel block: with many of
    them and few rows two kernels are faster, with few of them one is (a workspace
    without hidden rows tells which is taken)."""
    import submanifold_sparse_convolution_hash_amd as sc

    alone = sc.load_library().submconv_gated_ffn_inference_workspace_bytes
    one = [(9, 64, 256), (300, 64, 512), (4096, 64, 2048), (300, 128, 64), (300, 128, 256), (8192, 128, 2048),
           (20000, 128, 512)]
    two = [(9, 64, 2048), (300, 64, 1024), (1000, 64, 2048), (300, 128, 512), (4000, 128, 1024), (9, 128, 2048)]
    for n, c, f in one:
        assert alone(n, c, f, c, 1) == 0, (n, c, f)
    for n, c, f in two:
        assert alone(n, c, f, c, 1) >= n * f * 2, (n, c, f)
