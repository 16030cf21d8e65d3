"""The merge of a tree's split records, bit for bit bi_attention on each node's own path: few and many rows, more than 32
full splits, groups of 64 q heads, and the most lanes behind a context."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from gpu_util import same_bits
from tree_util import Case, make_tree

pytestmark = pytest.mark.gpu


def _many(c):
    """More rows x heads than 16 an SM: the merge that holds few records ahead."""
    return c.T * c.hq > 16 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("hq,hkv,hd,n,split,starts,many", [
    (16, 1, 64, 44, 64, [2050, 2111, 2559, 2700], True),      # 32 to 42 full splits
    (32, 1, 128, 27, 128, [1000, 1279, 700], True),           # 5 to 9
    (32, 1, 128, 27, 512, [2047, 2559, 1100], True),          # 2 to 4
    (64, 2, 64, 20, 64, [2048, 4200, 63], True),              # up to 65
    (4, 2, 64, 3, 64, [2047, 2048, 2112, 4161], False),
    (8, 2, 128, 2, 64, [2049, 6500], False),                  # up to 101
    (2, 1, 128, 5, 512, [8191, 17000], False),                # up to 33
])
def test_every_split_is_merged_in_order(hq, hkv, hd, n, split, starts, many):
    rng = np.random.default_rng(n + split)
    c = Case([make_tree(("levels", "random")[b % 2], n, rng) for b in range(len(starts))], starts, hq, hkv, hd, seed=n,
             qscale=2.0)
    assert _many(c) == many
    assert same_bits(c.run(split=split), c.linear(split=split))
    assert bi.bi_device_status() == bi.BI_OK


@pytest.mark.parametrize("hq,hkv,hd", [(64, 1, 64), (64, 1, 128), (128, 2, 64)])
@pytest.mark.parametrize("n", [1, 9, 34])
def test_groups_of_64_heads(hq, hkv, hd, n):
    rng = np.random.default_rng(hd + n)
    starts = [0, 70, 509, 1100]
    c = Case([make_tree(("chain", "levels")[b % 2], n, rng) for b in range(4)], starts, hq, hkv, hd, seed=hd)
    assert same_bits(c.run(), c.linear())


@pytest.mark.parametrize("hq,hkv,hd", [(2, 1, 64), (4, 2, 128)])
@pytest.mark.parametrize("split,start", [(832, 767), (832, 700), (832, 1599), (64, 127), (320, 255), (576, 1151)])
def test_the_longest_runs_of_lanes_behind_the_context(hq, hkv, hd, split, start):
    # 256 nodes on one path, from the last positions of a lane (832: lanes of 256, 256, 256 and 64)
    rng = np.random.default_rng(split)
    c = Case([make_tree("chain", 256, rng), make_tree("levels", 90, rng)], [start, start - 1], hq, hkv, hd, seed=start)
    assert same_bits(c.run(split=split), c.linear(split=split))
    assert bi.bi_device_status() == bi.BI_OK
