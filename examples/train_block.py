"""Fits one residual block (convolution, layer norm, gated feed-forward) to a
target on the sites of a sphere's shell, then runs it without gradients.

    python examples/train_block.py [--grid 48] [--channels 64] [--steps 20]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import submanifold_sparse_convolution_hash_amd as sc  # noqa: E402
from submanifold_sparse_convolution_hash_amd.blocks import SparseConvBlock  # noqa: E402


def sphere(grid: int, device) -> torch.Tensor:
    """Sites (0, x, y, z) within one voxel of a sphere of radius 0.4 grid."""
    r = torch.arange(grid, device=device, dtype=torch.float32) - (grid - 1) / 2
    d = (r[:, None, None] ** 2 + r[None, :, None] ** 2 + r[None, None, :] ** 2).sqrt()
    xyz = ((d - 0.4 * grid).abs() < 1).nonzero()
    return torch.cat([torch.zeros_like(xyz[:, :1]), xyz], 1).to(torch.int32).contiguous()


def train(grid: int = 48, channels: int = 64, steps: int = 20, device: str = "cuda"):
    """The loss of every step, and the trained block's inference error."""
    dev = torch.device(device, 0)
    torch.manual_seed(0)
    coords = sphere(grid, dev)
    n = coords.shape[0]
    kmap = sc.build_map(coords, (grid, grid, grid), 1)
    x = torch.randn(n, 8, device=dev).half()
    pos = coords[:, 1:].float() / grid
    target = torch.sin(pos @ torch.randn(3, channels, device=dev) * 6).half()
    block = SparseConvBlock(channels, 4 * channels, cin=8, device=dev)
    params = list(block.parameters())
    master = [p.detach().float().clone() for p in params]
    opt = torch.optim.Adam(master, lr=3e-3)
    scale = 1024.0  # keeps small fp16 gradients above the smallest numbers
    losses = []
    for _ in range(steps):
        out = block(kmap, x)
        loss = (out.float() - target.float()).square().mean()
        (loss * scale).backward()
        for p, m in zip(params, master):
            m.grad = p.grad.float() / scale
            p.grad = None
        opt.step()
        with torch.no_grad():
            for p, m in zip(params, master):
                p.copy_(m)
        losses.append(float(loss.detach()))
    with torch.no_grad():
        final = float((block(kmap, x).float() - target.float()).square().mean())
    kmap.free()
    return losses, final


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--grid", type=int, default=48)
    ap.add_argument("--channels", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, final = train(a.grid, a.channels, a.steps)
    for i, v in enumerate(losses):
        print(f"step {i:3d}  loss {v:.4f}")
    print(f"inference loss {final:.4f}")
