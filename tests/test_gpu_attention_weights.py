"""The fp16 forward's weights: small ones beside a large one.

One key leads all others by `gap` and has value 0, the others have equal scores
and values of about 1, so that the output is what the small weights carry. With u
= 2^-11, v = 2^-24 and p the weights, an output is off by at most
- a rounding of each weight to 16 bits: u p |v|, and below the smallest normal
  number half of a step, 2^-25, at a scale that has the largest weight at 2^7 or
  above: 2^-32 |v|;
- the fp32 sums of all keys, above and below the line: (keys + 32) v p |v| each;
- exponents, which are exact products here but for log2(e)'s and the difference's
  rounding, 2 v |gap| log2(e) each, and exp2 itself: 128 v p |v| for gaps below 18;
- the stored value's rounding: u |out|, or half a subnormal step, 2^-25.
"""
import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
U, V = 2.0 ** -11, 2.0 ** -24

# rows, keys, heads, key heads, columns
SHAPES = [
    (1, 2 ** 17, 4, 1, 64),     # a token over a long cache: one wave, the keys split
    (3, 4097, 2, 2, 128),
    (100, 2 ** 17 + 5, 1, 1, 32),  # four waves, the keys split
    (1500, 1473, 2, 2, 32),     # two groups of waves
    (20000, 1000, 2, 2, 64),    # four waves, one run
]


@gpu
@pytest.mark.parametrize("gap", [16.234375, 17.40625])
@pytest.mark.parametrize("shape", SHAPES)
def test_small_weights_beside_a_large_one(shape, gap):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import submanifold_sparse_convolution_hash_amd as sc

    rows, keys, heads, kv_heads, d = shape
    dev = torch.device("cuda:0")
    q = torch.zeros((rows, heads, d), dtype=torch.float16, device=dev)
    k = torch.zeros((keys, kv_heads, d), dtype=torch.float16, device=dev)
    q[:, :, 0] = 1.0
    k[0, :, 0] = gap
    gen = torch.Generator().manual_seed(keys)
    v = (1 + 0.25 * torch.randn((keys, kv_heads, d), generator=gen)).half()
    v[0] = 0.0
    out, lse = sc.attention(q, k, v.to(dev), scale=1.0, return_lse=True)
    small = np.exp(-gap)
    total = 1 + (keys - 1) * small
    one = np.abs(v.double().numpy()).sum(0), v.double().numpy().sum(0)  # [key heads][columns]
    size, ref = (np.repeat(t, heads // kv_heads, 0)[None] for t in one)
    ref = ref * small / total
    tol = size * small / total * (U + 2 * (keys + 32) * V + 128 * V) + 2.0 ** -32 * size + U * np.abs(ref) + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"{(err / tol).max():.3g} x the bound, out {out[0, 0, 0].item():.3g} of {ref[0, 0, 0]:.3g}"
    want = gap + np.log(total)
    assert np.abs(lse.double().cpu().numpy() - want).max() <= (keys + 64) * V + 8 * V * want


@gpu
def test_weights_that_grow_by_less_than_the_slack_stay_finite():
    """Scores that rise tile by tile, each step just below what raises the running
    maximum, from 2^7 on: the weights stay in fp16's range, up to its last
    power of two. Values are 1, so out is 1 up to the roundings above."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import submanifold_sparse_convolution_hash_amd as sc

    dev = torch.device("cuda:0")
    for rows, keys, d in ((1, 1280, 64), (200, 1280, 32), (1500, 1473, 128)):
        q = torch.zeros((rows, 1, d), dtype=torch.float16, device=dev)
        k = torch.zeros((keys, 1, d), dtype=torch.float16, device=dev)
        q[:, 0, 0] = 1.0
        for step in (5.53125, 5.546875, 8.0, 0.6875):  # 8 powers of two are 5.545
            k[:, 0, 0] = (torch.arange(keys, device=dev) // 64 * step).half()
            v = torch.ones_like(k)
            out, lse = sc.attention(q, k, v, scale=1.0, return_lse=True)
            want = torch.logsumexp(k[:, 0, 0].double(), 0).item()
            assert (out.double() - 1).abs().max().item() <= 2 * U + 2 * (keys + 32) * V + keys * 2.0 ** -32
            assert (lse.double() - want).abs().max().item() <= (keys + 64) * V + 8 * V * want
