"""A rollout on a pool of cache blocks that cannot hold it is refused before any block is taken."""
import numpy as np
import pytest
import torch

from invariant_forward_policy_gb300.decoder import Decoder, KVCache, KVPool
from oracle import paging


def _pool(B, mb, nb, owned=None, head=0):
    """A pool on the host whose sequence b holds owned[b] blocks."""
    pool = KVPool(B, mb, nb, device="cpu")
    owned = [0] * B if owned is None else owned
    held = sum(owned)
    pool.owned.copy_(torch.tensor(owned))
    ids = list(range(nb))
    for b in range(B):
        for j in range(owned[b]):
            pool.table[b, j] = ids.pop()
    for i, v in enumerate(ids):
        pool.ring[(head + i) % nb] = v
    pool.pool.copy_(torch.tensor([head, nb - held]))
    return pool


def _refused(pool, lens, n_gen, match):
    before = [t.clone() for t in (pool.table, pool.owned, pool.ring, pool.pool)]
    dec = object.__new__(Decoder)
    dec.device = torch.device("cpu")
    with pytest.raises(ValueError, match=match):
        dec.rollout([[1] * n for n in lens], n_gen, KVCache(None, None, pool.n_blocks), None, pool=pool)
    assert all(torch.equal(a, b) for a, b in zip(before, (pool.table, pool.owned, pool.ring, pool.pool)))


def test_short_pools_are_refused():
    _refused(_pool(2, 4, 3), [64, 65], 2, "blocks")           # 2 + 2 blocks of 3
    _refused(_pool(2, 4, 3), [60, 65], 6, "blocks")           # 1 + 2 for the prompts, the fourth in the last step
    _refused(_pool(2, 4, 9, owned=[4, 4]), [1, 150], 140, "blocks")  # 3 + 5 of at most 4
    _refused(_pool(2, 4, 5, owned=[0, 4]), [129, 1], 2, "blocks")    # request 1's come back too late for the first call
    _refused(_pool(2, 4, 5, owned=[4, 1]), [1, 200], 50, "blocks")
    _refused(_pool(1, 2, 2), [64], 65, "blocks")              # 128 positions are written, but the decode step asks
                                                              # for a table of 129


def test_damaged_pools_are_refused():
    for at, bad in (("pool", [5, 1]), ("pool", [-1, 1]), ("pool", [0, 6]), ("pool", [0, -1]), ("owned", [-1, 0]),
                    ("owned", [5, 0]), ("owned", [1, 1])):    # the last: seven blocks of five
        pool = _pool(2, 4, 5)
        getattr(pool, at).copy_(torch.tensor(bad))
        _refused(pool, [3, 4], 2, "pool")


def test_what_the_check_lets_through_is_served():
    """Random pools against the planning oracle run step by step: served throughout iff the check says so."""
    rng = np.random.default_rng(3)
    outcomes = [0, 0]
    for _ in range(300):
        B, mb = int(rng.integers(1, 5)), int(rng.integers(2, 6))
        owned = [int(v) for v in rng.integers(0, mb + 1, B)]
        nb = sum(owned) + int(rng.integers(0, 2 * B + 3))
        if nb == 0:
            continue
        pool = _pool(B, mb, nb, owned, head=int(rng.integers(0, nb)))
        n_gen = int(rng.integers(1, 90))
        lens = rng.integers(1, max(2, mb * 64 - n_gen + 1), B)
        if lens.max() + n_gen > mb * 64:
            continue
        head, count = pool.pool.tolist()
        table, own, free = pool.table.tolist(), list(owned), [pool.ring[(head + i) % nb].item() for i in range(count)]
        failed = False
        for step in range(n_gen):
            table, own, free, bad = paging.resize([int(n) + max(0, step - 1) for n in lens], min(step, 1), table, own,
                                                  free)
            failed = failed or bool(bad)
        try:
            pool.check([int(n) for n in lens], [int(n) + n_gen - 1 for n in lens])
            refused = False
        except ValueError:
            refused = True
        assert refused == failed, (owned, nb, lens, n_gen)
        outcomes[failed] += 1
    assert min(outcomes) > 20                                 # both happen
