"""A training step of the attention block, captured into a graph and replayed with
other inputs between eager work: bit for bit what eager steps give."""
import pytest
import torch

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("lengths", [[40, 0, 90], [700, 900]])
def test_captured_training_step(lengths):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import submanifold_sparse_convolution_hash_amd as sc

    dev = torch.device("cuda:0")
    torch.manual_seed(5)
    m = sc.SparseAttentionBlock(64, 96, heads=4, kv_heads=2, groups=8, context=24, rotary=12, device=dev)
    params = list(m.parameters())
    n, items = sum(lengths), len(lengths)
    off = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).to(dev)
    coff = (torch.arange(items + 1) * 5).to(torch.int32).to(dev)
    at = torch.randint(0, 64, (n, 3), device=dev, dtype=torch.int32)
    xs = [torch.randn(n, 64, device=dev).half() for _ in range(3)]
    ctx = torch.randn(5 * items, 24, device=dev).half()
    g = torch.randn(n, 64, device=dev).half()

    def step(x):
        y = m(x, off, at, ctx, coff)
        return [y, *torch.autograd.grad(y, [x, *params], g)]

    want = [[t.detach().clone() for t in step(x.clone().requires_grad_())] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm, and no eager graph of the parameters lives on
        step(xs[0].clone().requires_grad_())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    x = xs[0].clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    for turn in range(6):
        with torch.no_grad():
            x.copy_(xs[turn % 3])
        graph.replay()
        with torch.no_grad():
            eager = m(xs[1], off, at, ctx, coff)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[turn % 3])), turn
        assert torch.isfinite(eager.float()).all()
