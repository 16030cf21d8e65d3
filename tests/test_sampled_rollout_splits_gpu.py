"""A rollout whose decode steps share each logit row over eight CTAs, against a recompute that gives a
row to one CTA and another that shares it by two and four: the same bits."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300.decoder import Decoder
from synthetic import DecoderShape, make_decoder_weights, make_prompts
from tests.gpu_util import same_bits

pytestmark = pytest.mark.gpu


def test_decode_and_recompute_split_rows_differently():
    # three rows of 20000 logits: 8 CTAs each; 210 rows in one pass: one; 100 and 60 rows: two and four
    shape = DecoderShape(2, 128, 4, 2, 64, 256, 20000)
    dec = Decoder(shape, make_decoder_weights(shape, seed=91, w_std=0.05), max_pos=512)
    B, mb, n_gen = 3, 4, 70
    prompts = make_prompts(B, 10, 90, shape.vocab, seed=92)
    bt = dec.block_table(B, mb, seed=6)
    u = torch.rand((n_gen, B), generator=torch.Generator(device="cuda").manual_seed(93), device="cuda")
    f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    for rules in (bi.bi_sampling(f([0.8, 1.0, 1.3])),
                  bi.bi_sampling(f([0.9, 1.1, 1.0]), torch.tensor([40, 0, 900], dtype=torch.int32, device="cuda"),
                                 f([0.95, 0.9, 1.0]), f([0.0, 0.0, 0.01]))):
        ids, lp = dec.rollout(prompts, n_gen, dec.alloc_cache(B * mb), bt, sampling=rules, uniforms=u)
        assert torch.isfinite(lp).all()
        gens = ids.cpu().numpy()
        for rows in (2048, 100, 60):
            got = dec.recompute(prompts, gens, dec.alloc_cache(B * mb), bt, sampling=rules, max_logit_rows=rows)
            assert same_bits(got, lp), rows
        assert np.unique(gens).size > 50
    assert bi.bi_device_status() == 0
