"""Infinite and NaN keys and values before the tree: a row has what bi_attention gives on its path, whether they fill a key, a
lane, a split or the whole context."""
import numpy as np
import pytest
import torch

from tree_util import Case, make_tree

pytestmark = pytest.mark.gpu


def _same(a, b):
    nan = torch.isnan(a)
    return torch.equal(nan, torch.isnan(b)) and torch.equal(a[~nan].view(torch.int16), b[~nan].view(torch.int16))


@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (8, 1, 128), (32, 1, 64)])
@pytest.mark.parametrize("where", [(130, 131), (500, 514), (128, 256), (512, 1024), (0, 1300), (1280, 1300), (0, 1303)])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf, 3e38])
@pytest.mark.parametrize("of", ["k", "v"])
def test_poisoned_context(hq, hkv, hd, where, what, of):
    rng = np.random.default_rng(hd + where[0])
    c = Case([make_tree("levels", 24, rng), make_tree("random", 60, rng)], [1300, 600], hq, hkv, hd, seed=hq)
    c.q[::2] = np.abs(c.q[::2]) + 0.1          # scores of one sign on infinite keys, and of both
    getattr(c, of)[0][where[0]:where[1]] = what
    assert _same(c.run(), c.linear())
