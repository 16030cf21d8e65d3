"""Acceptance where a sequence's positions end: the next start is a 32-bit position or the sequence accepts nothing."""
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from tree_util import i32

pytestmark = pytest.mark.gpu

TOP = 2**31 - 1


@pytest.mark.parametrize("start,fits", [(TOP - 3, True), (TOP - 2, False), (TOP, False)])
def test_a_start_near_the_last_position(start, fits):
    # two sequences of the chain 4 -> 5 -> 6, all chosen; the first stands far from the end
    parent, tokens, targets = i32([-1, 0, 1] * 2), i32([4, 5, 6] * 2), i32([5, 6, 7] * 2)
    count, pos = i32([-9, -9]), i32([-9, -9])
    path, out = i32([[-9] * 3] * 2), i32([[-9] * 3] * 2)
    bi.bi_tree_accept(parent, i32([0, 3, 6]), i32([100, start]), tokens, targets, 2, 3, 6, 3, count, path, out, pos)
    assert bi.bi_device_status() == (bi.BI_OK if fits else bi.BI_ERR_DEVICE_CHECK)
    assert count.tolist() == [3, 3 if fits else 0] and pos.tolist() == [103, start + 3 if fits else start]
    assert path.tolist() == [[0, 1, 2], [0, 1, 2] if fits else [-1] * 3]
    assert out.tolist() == [[5, 6, 7], [5, 6, 7] if fits else [-1] * 3]


def test_a_sequence_without_nodes_at_the_last_position():
    count, pos, path, out = i32([-9]), i32([-9]), i32([[-9]]), i32([[-9]])
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    bi.bi_tree_accept(none, i32([0, 0]), i32([TOP]), none, none, 1, 1, 1, 1, count, path, out, pos)
    assert bi.bi_device_status() == bi.BI_OK and count.tolist() == [0] and pos.tolist() == [TOP]
