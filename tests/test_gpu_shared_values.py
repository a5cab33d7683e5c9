"""attend_shared where bf16 values are so large that a running maximum may not lag far behind."""

import pytest
import torch

from test_gpu_shared import BF16, ns, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,mask", [(1, 4, None), (9, 8, "tree"), (20, 16, "tree")])
def test_large_values_behind_keys_that_come_to_count_late(ns, d, n, hq, mask):  # noqa: F811
    """Values of about 2^104 in bf16, and scores that grow eightfold behind the first two tiles: by a maximum of those,
    probabilities of 2^24 and more come to sums beyond fp32, whose final sizes are far below.  By a maximum that leaves 64
    probabilities at most 2^15, the 16 times 64 keys have sums of at most 16 * 2^15 * 2^107 = 2^126: within it.
    24 groups on 4 heads, so that a block has several tiles of an item.  The tolerance is that of any other values."""
    def spoil(k, v, row):
        v.mul_(2.0 ** 104)
        for b in range(0, 48, 2):
            at = [row(b, p) for p in range(256, 900)]
            k[[i for i, _ in at], :, [r for _, r in at]] *= 8
        assert v.abs().max() < 2.0 ** 107
    run(ns, [910] * 24, [[n, n + 5]] * 24, n, hq, 4, d, BF16, 16, d + n, mask, spoil=spoil)
