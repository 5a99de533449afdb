"""Fits one attention block (group norm, attention among an item's sites with
rotary coordinates, attention over a few rows of conditioning, gated
feed-forward) to a target on the sites of two spheres' shells.

    python examples/train_attention.py [--grid 24] [--channels 64] [--steps 20]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import submanifold_sparse_convolution_hash_amd as sc  # noqa: E402


def spheres(grid: int, device) -> torch.Tensor:
    """Sites (b, x, y, z) within one voxel of spheres of radius 0.4 and 0.3 grid."""
    r = torch.arange(grid, device=device, dtype=torch.float32) - (grid - 1) / 2
    d = (r[:, None, None] ** 2 + r[None, :, None] ** 2 + r[None, None, :] ** 2).sqrt()
    shells = [((d - k * grid).abs() < 1).nonzero() for k in (0.4, 0.3)]
    return torch.cat([torch.nn.functional.pad(s, (1, 0), value=b) for b, s in enumerate(shells)]).to(torch.int32)


def train(grid: int = 24, channels: int = 64, steps: int = 20, device: str = "cuda"):
    """The loss of every step, and the trained block's inference error."""
    dev = torch.device(device, 0)
    torch.manual_seed(0)
    coords = spheres(grid, dev)
    offsets = sc.item_offsets(coords, 2)
    positions = coords[:, 1:]
    x = torch.randn(coords.shape[0], channels, device=dev).half()
    context = torch.randn(2 * 5, 32, device=dev).half()
    context_offsets = torch.tensor([0, 5, 10], dtype=torch.int32, device=dev)
    target = torch.sin(positions.float() / grid @ torch.randn(3, channels, device=dev) * 6).half()
    turned = channels // 4 // 6 * 6  # columns of a head: pairs for three axes
    block = sc.SparseAttentionBlock(channels, 4 * channels, heads=4, kv_heads=2, groups=8, context=32, rotary=turned,
                                    device=dev)
    params = list(block.parameters())
    master = [p.detach().float().clone() for p in params]
    opt = torch.optim.Adam(master, lr=3e-3)
    scale = 1024.0  # keeps small fp16 gradients above the smallest numbers
    losses = []
    for _ in range(steps):
        out = block(x, offsets, positions, context, context_offsets)
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
        final = float((block(x, offsets, positions, context, context_offsets).float() - target.float()).square().mean())
    return losses, final


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--grid", type=int, default=24)
    ap.add_argument("--channels", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, final = train(a.grid, a.channels, a.steps)
    for i, v in enumerate(losses):
        print(f"step {i:3d}  loss {v:.4f}")
    print(f"inference loss {final:.4f}")
