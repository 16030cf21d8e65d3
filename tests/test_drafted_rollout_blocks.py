"""A drafted rollout needs blocks for every sequence's own drafts: a table that lacks them is refused before it starts."""
import numpy as np
import pytest
import torch

from invariant_forward_policy_gb300.decoder import Decoder, KVCache, paged_block_ids
from synthetic import DecoderShape


class Started(Exception):
    pass


def _run(lens, n_gen, max_nodes, table, n_blocks):
    dec = object.__new__(Decoder)
    dec.shape, dec.device, dec.fp8, dec.max_pos = DecoderShape(1, 128, 4, 2, 64, 256, 512), torch.device("cpu"), False, 4096

    def prefill(*args, **kw):
        raise Started
    dec.prefill = prefill
    dec.rollout_drafted([[1] * n for n in lens], n_gen, KVCache(None, None, n_blocks), torch.from_numpy(table),
                        lambda b, tokens: ([], []), max_nodes=max_nodes)


def test_a_ragged_table_for_the_plain_rollout_lacks_the_drafts_blocks():
    lens, n_gen, max_nodes = np.array([300, 61, 100]), 4, 8
    plain, nb = paged_block_ids(lens + n_gen - 1, 6, 3)
    with pytest.raises(ValueError, match="sequence 1"):       # 71 positions, one block; the others fit in their last ones
        _run(lens, n_gen, max_nodes, plain, nb)
    drafted, nb = paged_block_ids(lens + n_gen + max_nodes - 2, 6, 3)
    with pytest.raises(Started):
        _run(lens, n_gen, max_nodes, drafted, nb)


@pytest.mark.parametrize("at,bad", [((0, 2), -1), ((1, 0), -1), ((1, 1), 9), ((0, 0), 1 << 30)])
def test_entries_that_are_no_block_of_the_cache(at, bad):
    table = np.arange(9, dtype=np.int32).reshape(3, 3)        # 129 and 65 positions of two sequences, and a third's row
    args = [122, 58], 5, 4
    with pytest.raises(Started):
        _run(*args, table, 9)
    table[at] = bad
    with pytest.raises(ValueError, match=f"sequence {at[0]}"):
        _run(*args, table, 9)


def test_entries_that_no_position_reaches_do_not_matter():
    table = np.array([[0, 1, 2], [3, -1, -1]], np.int32)
    with pytest.raises(Started):
        _run([122, 57], 5, 4, table, 4)
    with pytest.raises(ValueError, match="sequences"):
        _run([122, 57, 3], 5, 4, table, 4)
