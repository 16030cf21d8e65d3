"""Drafted rollouts end to end: trees of drafts that are right, wrong or both, greedy and sampled, give the plain
rollout's tokens and logprobs bit for bit, and the recompute's scores of them."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300.decoder import Decoder
from synthetic import DecoderShape, make_decoder_weights, make_prompts
from tests.gpu_util import same_bits

pytestmark = pytest.mark.gpu


def _drafter(ids, prompts, vocab, seed, right=0.8):
    """Trees around the true continuation: a path of it, broken with probability 1 - right a token, and side branches."""
    rng = np.random.default_rng(seed)
    calls = []

    def draft(b, tokens):
        done = len(tokens) - len(prompts[b])
        assert tokens[len(prompts[b]):].tolist() == ids[b, :done].tolist()
        calls.append(b)
        toks, pars, at = [], [], -1
        for t in ids[b, done:done + int(rng.integers(0, 9))]:
            for _ in range(int(rng.integers(0, 3))):        # wrong siblings before and after the right one
                toks.append(int(rng.integers(0, vocab)))
                pars.append(at)
            toks.append(int(t) if rng.random() < right else int(rng.integers(0, vocab)))
            pars.append(at)
            at = len(toks) - 1
            if rng.random() < 0.3:
                toks.append(int(rng.integers(0, vocab)))
                pars.append(at)
        return toks, pars
    draft.calls = calls
    return draft


@pytest.mark.parametrize("shape,B,lo,hi,n_gen", [
    (DecoderShape(2, 128, 4, 2, 64, 256, 2048), 5, 10, 150, 40),
    (DecoderShape(2, 256, 4, 4, 64, 512, 512), 3, 480, 540, 30),          # across a split
    (DecoderShape(2, 512, 8, 2, 128, 512, 1024, kv_split=128), 2, 60, 200, 70),
])
@pytest.mark.parametrize("sampled", [False, True])
def test_drafted_rollout_equals_rollout(shape, B, lo, hi, n_gen, sampled):
    dec = Decoder(shape, make_decoder_weights(shape, seed=71, w_std=0.05), max_pos=1024)
    prompts = make_prompts(B, lo, hi, shape.vocab, seed=72)
    max_nodes = 24
    mb = -(-(max(len(p) for p in prompts) + n_gen + max_nodes) // 64)
    bt = dec.block_table(B, mb, seed=4)
    kw = {}
    if sampled:
        temp = torch.linspace(0.5, 1.2, B, device="cuda")
        kw = dict(sampling=bi.bi_sampling(temp, torch.full((B,), 40, dtype=torch.int32, device="cuda"),
                                          torch.full((B,), 0.95, device="cuda")),
                  uniforms=torch.rand((n_gen, B), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda"))
    ids, lp = dec.rollout(prompts, n_gen, dec.alloc_cache(B * mb), bt, **kw)
    want = ids.cpu().numpy()
    none = lambda b, tokens: ([], [])
    for draft in (_drafter(want, prompts, shape.vocab, 5), _drafter(want, prompts, shape.vocab, 6, right=1.0), none):
        got, glp = dec.rollout_drafted(prompts, n_gen, dec.alloc_cache(B * mb), bt, draft, max_nodes=max_nodes, **kw)
        assert torch.equal(got, ids) and same_bits(glp, lp)
        assert bi.bi_device_status() == bi.BI_OK
        if draft is not none:      # drafts save passes
            assert len(draft.calls) < B * (n_gen - 1) * 0.7
    score = dict(sampling=kw["sampling"]) if sampled else {}
    lp_t = dec.recompute(prompts, want, dec.alloc_cache(B * mb), bt, chunk=97, **score)
    assert same_bits(lp_t, lp)


def test_drafted_rollout_refusals():
    shape = DecoderShape(1, 128, 2, 2, 64, 256, 512)
    w = make_decoder_weights(shape, seed=71, w_std=0.05)
    dec = Decoder(shape, w, max_pos=128)
    prompts = make_prompts(2, 20, 30, shape.vocab, seed=72)
    cache, bt = dec.alloc_cache(4), dec.block_table(2, 2, seed=4)
    none = lambda b, tokens: ([], [])
    with pytest.raises(ValueError):
        dec.rollout_drafted(prompts, 8, cache, bt, none, max_nodes=257)
    with pytest.raises(ValueError):
        dec.rollout_drafted(prompts, 8, cache, bt, none, max_nodes=100)        # blocks
    with pytest.raises(ValueError):
        dec.rollout_drafted(prompts, 120, cache, bt, none, max_nodes=2)        # RoPE rows
    with pytest.raises(ValueError):
        dec.rollout_drafted(prompts, 8, cache, bt, none, uniforms=torch.zeros((8, 2), device="cuda"))
    with pytest.raises(ValueError):
        dec.rollout_drafted(prompts, 8, cache, bt, lambda b, t: ([1], [0]))
    with pytest.raises(ValueError):
        Decoder(shape, w, max_pos=128, fp8=True).rollout_drafted(prompts, 8, cache, bt, none)


def _step_case(n_nodes, extra, seed=81):
    shape = DecoderShape(2, 128, 4, 2, 64, 256, 512)
    dec = Decoder(shape, make_decoder_weights(shape, seed=71, w_std=0.05), max_pos=256)
    rng = np.random.default_rng(seed)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    parent = [int(rng.integers(0, i)) if i else -1 for n in n_nodes for i in range(n)] + [-1] * extra
    tokens = rng.integers(0, shape.vocab, len(parent)).tolist()
    cache = dec.alloc_cache(2 * len(n_nodes))
    for c in (cache.k, cache.v):
        c.copy_(torch.randn(c.shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
    return dec, i32(tokens), i32(parent), i32(n_nodes), i32([70] * len(n_nodes)), cache, dec.block_table(
        len(n_nodes), 2, seed=4)


def test_tree_step_rows_without_a_sequence_write_nothing():
    n_nodes, extra = [5, 0, 9], 6
    dec, tokens, parent, n, start, cache, bt = _step_case(n_nodes, extra)
    T = sum(n_nodes)
    before = cache.k.clone(), cache.v.clone()
    ids, lp, row0, pos = dec.tree_step(tokens[:T].clone(), parent[:T].clone(), n, start, 16, cache, bt, 100)
    assert bi.bi_device_status() == bi.BI_OK
    after = cache.k.clone(), cache.v.clone()
    cache.k.copy_(before[0])
    cache.v.copy_(before[1])
    # what the allocator hands out next holds valid slots and positions
    junk = [torch.full((T + extra,), 7, dtype=t, device="cuda") for t in (torch.int64, torch.int32) for _ in range(8)]
    del junk
    ids2, lp2, row02, pos2 = dec.tree_step(tokens, parent, n, start, 16, cache, bt, 100)
    assert bi.bi_device_status() != bi.BI_OK
    assert torch.equal(ids2[:T], ids) and same_bits(lp2[:T], lp) and torch.equal(row02, row0)
    assert torch.equal(pos2[:T], pos) and (pos2[T:] == -1).all()
    assert same_bits(cache.k, after[0]) and same_bits(cache.v, after[1])


def test_tree_step_without_nodes():
    dec, tokens, parent, n, start, cache, bt = _step_case([0, 0], 0)
    before = cache.k.clone()
    ids, lp, row0, pos = dec.tree_step(tokens, parent, n, start, 4, cache, bt, 100)
    assert ids.numel() == lp.numel() == pos.numel() == 0 and row0.tolist() == [0, 0, 0]
    assert same_bits(cache.k, before) and bi.bi_device_status() == bi.BI_OK


def test_tree_step_refusals():
    dec, tokens, parent, n, start, cache, bt = _step_case([5, 4], 0)
    ok = dict(tokens=tokens, parent=parent, n_nodes=n, start=start, max_nodes=8, cache=cache, block_table=bt, max_ctx=100)
    for bad in (dict(parent=parent[:-1]), dict(tokens=tokens.long()), dict(start=start[:1]), dict(block_table=bt[:1]),
                dict(parent=torch.stack([parent, parent], 1)[:, 0]), dict(block_table=torch.cat([bt, bt], 1)[:, :2]),
                dict(sampling=bi.bi_sampling(None, None, None)),
                dict(sampling=bi.bi_sampling(None, None, None), u=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            dec.tree_step(**{**ok, **bad})


def test_tree_step_captured_and_replayed():
    dec, tokens, parent, n, start, cache, bt = _step_case([5, 0, 9], 0)
    before = cache.k.clone(), cache.v.clone()
    other = (tokens + 17) % dec.shape.vocab
    want = dec.tree_step(other, parent, n, start, 16, cache, bt, 100)
    end = cache.k.clone(), cache.v.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = dec.tree_step(tokens, parent, n, start, 16, cache, bt, 100)
    tokens.copy_(other)
    for _ in range(2):
        cache.k.copy_(before[0])
        cache.v.copy_(before[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and same_bits(got[1], want[1])
        assert same_bits(cache.k, end[0]) and same_bits(cache.v, end[1])
    assert bi.bi_device_status() == bi.BI_OK
