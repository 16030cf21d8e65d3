"""Pins of the paged-cache planning oracle: hand-worked tables, block conservation, and slots against
the host bookkeeping that the decoder uses."""
import numpy as np

from invariant_forward_policy_gb300.decoder import paged_block_ids
from oracle import paging


def test_hand_worked_growth_release_and_shortage():
    table = [[7, -1, -1], [3, 4, -1], [-1, -1, -1], [9, -1, -1]]
    # 65 tokens need two blocks; 0 tokens none; 129 three (short of one: two are left after request 0); 64 one
    t, owned, free, failed = paging.resize([65, 0, 129, 64], 0, table, [1, 2, 0, 1], [20, 21, 22])
    assert t == [[7, 20, -1], [-1, -1, -1], [-1, -1, -1], [9, -1, -1]]
    assert owned == [2, 0, 0, 1] and free == [21, 22, 3, 4] and failed == [2]
    # a decode step: the 64th token is in place, the 65th needs a block; an idle request stays idle
    t, owned, free, failed = paging.resize([64, 0], 1, [[1, -1], [-1, -1]], [1, 0], [5, 6])
    assert t == [[1, 5], [-1, -1]] and owned == [2, 0] and free == [6] and not failed


def test_blocks_are_conserved():
    rng = np.random.default_rng(1)
    B, mb, nb = 12, 6, 50
    table, owned, free = [[-1] * mb for _ in range(B)], [0] * B, list(rng.permutation(nb))
    for _ in range(200):
        lens = [int(n) for n in rng.integers(0, mb * 64 + 1, B)]
        table, owned, free, failed = paging.resize(lens, 0, table, owned, free)
        held = [i for r, n in zip(table, owned) for i in r[:n]]
        assert sorted(held + list(free)) == list(range(nb))
        assert all(i == -1 for r, n in zip(table, owned) for i in r[n:])
        assert all(owned[b] == -(-lens[b] // 64) for b in range(B) if b not in failed)


def test_slots_follow_the_block_table():
    ctx = [130, 1, 64, 200]
    tab, _ = paged_block_ids(ctx, 4, seed=3)
    row0, rows = paging.slot_map([2, 1, 0, 70], [128, 0, 64, 130], tab.tolist(), 100)
    assert row0 == [0, 2, 3, 3, 73]
    assert rows[0] == (0, 128, int(tab[0, 2]) * 64) and rows[2] == (1, 0, int(tab[1, 0]) * 64)
    assert rows[3] == (3, 130, int(tab[3, 2]) * 64 + 2) and rows[-1] == (3, 199, int(tab[3, 3]) * 64 + 7)
    assert paging.slot_map([3], [63], [[5, -1]], 2) == ([0, 2], [(0, 63, 5 * 64 + 63), (0, 64, -1)])
