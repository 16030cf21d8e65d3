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
