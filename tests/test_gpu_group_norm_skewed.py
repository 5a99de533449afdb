"""Group norm of batches in which one item has nearly all rows, on both sides of the
rule by which the outputs' workgroups join their item's chunks themselves: the
checks and bounds of the other shapes."""
import pytest
import torch

import test_gpu_packed as packed

gpu = pytest.mark.gpu

# rows per item (and rows behind the last), channels, groups, columns of padding
SKEWED = [
    ([20] * 15 + [49700], 0, 96, 32, 0),      # joined there, forward and backward
    ([49700] + [20] * 15, 7, 320, 32, 0),     # backward alone
    ([20] * 99 + [48000, 0], 0, 320, 32, 3),  # the same, many items
    ([3] * 50 + [99000] + [3] * 49, 0, 320, 32, 0),  # neither
]


@gpu
@pytest.mark.parametrize("case", range(len(SKEWED)))
def test_group_norm_of_one_large_item_among_small_ones(case, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    monkeypatch.setattr(packed, "NORMS", SKEWED)
    packed.test_group_norm(torch.device("cuda:0"), case, torch.float16)
