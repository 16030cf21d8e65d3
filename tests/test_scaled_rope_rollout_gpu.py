"""Rollouts of a decoder whose caller has put a scaled table in its rope_table: plain, drafted and recomputed bits agree, on
ragged block tables that hold just the blocks each sequence needs."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300.decoder import Decoder
from synthetic import DecoderShape, make_decoder_weights, make_prompts
from tests.gpu_util import same_bits

pytestmark = pytest.mark.gpu

SCALINGS = {"linear": dict(factor=4.0), "base": dict(factor=3.0), "turns": dict(factor=8.0, orig_len=64.0, low=1.0, high=4.0),
            "dims": dict(factor=40.0, orig_len=64.0, low=1.0, high=32.0, amplitude=0.1 * np.log(40) + 1)}


@pytest.mark.parametrize("kind", sorted(SCALINGS))
@pytest.mark.parametrize("shape", [DecoderShape(2, 128, 4, 2, 64, 256, 1024), DecoderShape(1, 256, 4, 1, 128, 256, 512)])
def test_scaled_table_in_a_decoder(kind, shape):
    dec = Decoder(shape, make_decoder_weights(shape, seed=71, w_std=0.05), max_pos=512)
    prompts, n_gen, max_nodes = make_prompts(4, 30, 200, shape.vocab, seed=72), 24, 12
    lens = np.array([len(p) for p in prompts])
    mb = -(-(int(lens.max()) + n_gen + max_nodes) // 64)
    bt, nb = dec.paged_block_table(lens + n_gen + max_nodes - 2, mb, seed=5)
    plain_lp = dec.rollout(prompts, n_gen, dec.alloc_cache(nb), bt)[1]
    bi.bi_rope_scaled_table(dec.rope_table, 512, shape.head_dim, shape.rope_theta,
                            bi.bi_rope_scaling(getattr(bi, "BI_ROPE_" + kind.upper()), **SCALINGS[kind]))
    ids, lp = dec.rollout(prompts, n_gen, dec.alloc_cache(nb), bt)
    assert not same_bits(lp, plain_lp)
    want = ids.cpu().numpy()

    def draft(b, tokens):                       # the true continuation behind a wrong sibling, broken now and then
        done = len(tokens) - lens[b]
        toks = [1] + want[b, done:done + 7].tolist()
        if done % 3 == 0:
            toks[len(toks) // 2] ^= 1
        return toks, [-1, -1] + list(range(1, len(toks) - 1))
    got, glp = dec.rollout_drafted(prompts, n_gen, dec.alloc_cache(nb), bt, draft, max_nodes=max_nodes)
    assert torch.equal(got, ids) and same_bits(glp, lp)
    assert same_bits(dec.recompute(prompts, want, dec.alloc_cache(nb), bt, chunk=97), lp)
    assert bi.bi_device_status() == bi.BI_OK
