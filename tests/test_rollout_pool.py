"""A rollout on a pool of cache blocks that cannot hold it is refused before any block is taken."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
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


def test_prompts_without_a_token_are_refused():
    _refused(_pool(2, 4, 8), [3, 0], 4, "token")
    _refused(_pool(2, 4, 8), [3, 1], 0, "n_gen")
    dec = object.__new__(Decoder)
    dec.device = torch.device("cpu")
    for lens, n_gen, match in (([3, 0], 4, "token"), ([3, 1], 0, "n_gen")):
        with pytest.raises(ValueError, match=match):          # drawn without a pool
            dec.rollout([[1] * n for n in lens], n_gen, KVCache(None, None, 8), None, sampling=bi.bi_sampling(),
                        uniforms=torch.zeros(n_gen, 2))


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


def test_taken_blocks_are_put_back():
    """What `saved` and `restore` of a pool hold, on the host."""
    pool = _pool(2, 4, 9, owned=[1, 2], head=4)
    before = [t.clone() for t in (pool.table, pool.owned, pool.ring, pool.pool)]
    held = pool.saved()
    for t in (pool.table, pool.owned, pool.ring, pool.pool):
        t.fill_(-5)
    pool.restore(held)
    assert all(torch.equal(a, b) for a, b in zip(before, (pool.table, pool.owned, pool.ring, pool.pool)))


@pytest.mark.gpu
@pytest.mark.parametrize("sampled", [False, True])
def test_a_refused_call_gives_its_blocks_back(sampled):
    """Arguments that the forward calls refuse: the pool is as it was, and serves the corrected call."""
    from synthetic import DecoderShape, make_decoder_weights, make_prompts
    from tests.gpu_util import same_bits
    shape = DecoderShape(2, 128, 4, 2, 64, 256, 2048)
    dec = Decoder(shape, make_decoder_weights(shape, seed=81, w_std=0.05), max_pos=256)
    B, mb, n_gen = 3, 4, 9
    prompts = make_prompts(B, 30, 120, shape.vocab, seed=82)
    u = torch.rand((n_gen, B), generator=torch.Generator(device="cuda").manual_seed(83), device="cuda")
    kw = dict(sampling=bi.bi_sampling(), uniforms=u) if sampled else {}
    pool = KVPool(B, mb, B * mb, seed=5)
    pool.resize(torch.tensor([70, 0, 10], dtype=torch.int32, device="cuda"))
    before = [t.clone() for t in (pool.table, pool.owned, pool.ring, pool.pool)]
    cache = dec.alloc_cache(B * mb)
    bad = [dict(chunk=0), dict(prefill_max_tokens=0), dict(mode=7)]
    if sampled:
        bad.append(dict(sampling=bi.bi_sampling(torch.ones(B - 1, device="cuda"))))
        bad.append(dict(uniforms=u.cpu()))
    for b in bad:
        with pytest.raises(Exception):
            dec.rollout(prompts, n_gen, cache, None, pool=pool, **{**kw, **b})
        assert all(torch.equal(a, c) for a, c in zip(before, (pool.table, pool.owned, pool.ring, pool.pool))), b
    wide = KVPool(1, 8, 8)                                    # past max_pos in the model, not in the table
    with pytest.raises(Exception):
        dec.rollout([[1] * 270], 1, cache, None, pool=wide)
    assert wide.pool.cpu().tolist() == [0, 8] and wide.owned.item() == 0 and (wide.table == -1).all()
    ids, lp = dec.rollout(prompts, n_gen, cache, None, pool=pool, **kw)
    bt = dec.block_table(B, mb, seed=4)
    ids_t, lp_t = dec.rollout(prompts, n_gen, dec.alloc_cache(B * mb), bt, **kw)
    assert torch.equal(ids, ids_t) and same_bits(lp, lp_t)
    assert bi.bi_device_status() == 0
