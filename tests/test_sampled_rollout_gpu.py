"""Sampled rollouts end to end: drawn tokens and their logprobs in graph and eager decode, with block
tables grown on the device, against the recompute's scores of the same tokens, bit for bit."""
import math

import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300.decoder import Decoder, KVPool
from synthetic import DecoderShape, make_decoder_weights, make_prompts
from tests.gpu_util import dev_bf16_from_f32, same_bits

pytestmark = pytest.mark.gpu


def _rules(B, seed):
    """One rule per sequence: greedy, plain, and every cut."""
    rng = np.random.default_rng(seed)
    temp = rng.uniform(0.6, 1.4, B).astype(np.float32)
    temp[0] = 0.0
    k = np.array([0, 0, 20, 0, 5, 0, 1500][:B], np.int32)
    p = np.array([1, 1, 1, 0.9, 0.8, 1, 0.95][:B], np.float32)
    mp = np.array([0, 0, 0, 0, 0, 0.02, 0][:B], np.float32)
    return bi.bi_sampling(*(torch.from_numpy(a).cuda() for a in (temp, k, p, mp)))


@pytest.mark.parametrize("fp8", [False, True])
def test_sampled_rollout_equals_recompute(fp8):
    shape = DecoderShape(2, 128, 4, 2, 64, 256, 2048)
    dec = Decoder(shape, make_decoder_weights(shape, seed=61, w_std=0.05), max_pos=1024, fp8=fp8)
    B, n_gen = 7, 40
    prompts = make_prompts(B, 10, 150, shape.vocab, seed=62)
    mb = -(-(max(len(p) for p in prompts) + n_gen) // 64)
    rules = _rules(B, 63)
    u = torch.rand((n_gen, B), generator=torch.Generator(device="cuda").manual_seed(64), device="cuda")
    cache = dec.alloc_cache(B * mb)
    bt = dec.block_table(B, mb, seed=4)
    ids, lp = dec.rollout(prompts, n_gen, cache, bt, sampling=rules, uniforms=u)
    assert bi.bi_device_status() == 0
    ids_e, lp_e = dec.rollout(prompts, n_gen, dec.alloc_cache(B * mb), bt, use_graph=False, sampling=rules, uniforms=u)
    assert torch.equal(ids, ids_e) and same_bits(lp, lp_e)
    # blocks taken from a pool as the sequences grow: other pages, the same tokens; only what is needed is taken
    pool = KVPool(B, mb, B * mb, seed=9)
    ids_p, lp_p = dec.rollout(prompts, n_gen, dec.alloc_cache(B * mb), None, sampling=rules, uniforms=u, pool=pool)
    assert torch.equal(ids, ids_p) and same_bits(lp, lp_p)
    need = [-(-(len(p) + n_gen - 1) // 64) for p in prompts]
    assert pool.owned.cpu().tolist() == need
    assert bi.bi_device_status() == 0
    # the same distributions in the recompute: other packings and chunks, the same bits
    gens = ids.cpu().numpy()
    for chunk, order in ((2048, None), (64, [4, 2, 0, 6, 1, 3, 5]), (97, [6, 5, 4, 3, 2, 1, 0])):
        lp_t = dec.recompute(prompts, gens, dec.alloc_cache(B * mb), bt, chunk=chunk, order=order, sampling=rules,
                             max_logit_rows=50)
        assert same_bits(lp_t, lp), (chunk, order)
    lp_t = dec.recompute(prompts, gens, dec.alloc_cache(B * mb), pool.table, sampling=rules)
    assert same_bits(lp_t, lp)
    # the greedy sequence is the greedy rollout's, with logprob 0; the others are not
    ids_g, _ = dec.rollout(prompts, n_gen, dec.alloc_cache(B * mb), bt)
    assert torch.equal(ids[0], ids_g[0]) and (lp[0] == 0).all()
    assert all(not torch.equal(ids[b], ids_g[b]) for b in range(1, B))
    # released: every block is back
    pool.resize(torch.zeros(B, dtype=torch.int32, device="cuda"))
    assert pool.pool[1].item() == B * mb and (pool.table == -1).all()
    assert sorted(pool.ring.cpu().tolist()) == list(range(B * mb))


def test_plain_temperature_scores_like_the_fused_head():
    """At temperature 1 with nothing cut, the sampled logprob is the model's log-softmax: the fused head gives
    the same number up to the rounding of two fp32 evaluations (2^-20 of |lp|, a dozen roundings each)."""
    shape = DecoderShape(2, 128, 4, 2, 64, 256, 2048)
    dec = Decoder(shape, make_decoder_weights(shape, seed=71, w_std=0.05), max_pos=512)
    prompts = make_prompts(3, 10, 90, shape.vocab, seed=72)
    mb, n_gen = 3, 16
    bt = dec.block_table(3, mb, seed=1)
    u = torch.rand((n_gen, 3), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    ids, lp = dec.rollout(prompts, n_gen, dec.alloc_cache(3 * mb), bt, sampling=bi.bi_sampling(), uniforms=u)
    want = dec.recompute(prompts, ids.cpu().numpy(), dec.alloc_cache(3 * mb), bt)
    assert ((lp - want).abs() <= 2.0 ** -20 * want.abs()).all()
    fast, lpf = dec.rollout(prompts, n_gen, dec.alloc_cache(3 * mb), bt, sampling=bi.bi_sampling(), uniforms=u,
                            mode=bi.BI_FAST)
    assert fast.min().item() >= 0 and torch.isfinite(lpf).all()
    assert bi.bi_device_status() == 0


def test_a_step_planned_on_the_device():
    """Block tables and row metadata made on the GPU from lengths alone drive the QKV projection and attention:
    decode rows, a prefill chunk and an idle request in one step give the bits of a whole prefill."""
    Hq, Hkv, hd, d = 4, 2, 64, 128
    B, mb, nb = 4, 5, 24
    lens = [130, 64, 200, 0]
    steps = [[129, 0, 70, 0], [1, 64, 130, 0]]               # new tokens of two steps
    gen = torch.Generator().manual_seed(3)
    w = dev_bf16_from_f32((torch.randn((Hq + 2 * Hkv) * hd, d, generator=gen) * 0.1).numpy())
    x = [dev_bf16_from_f32(torch.randn(n, d, generator=gen).numpy()) for n in lens]
    table = torch.empty((512, hd), dtype=torch.float32, device="cuda")
    bi.bi_rope_table(table, 512, hd)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(plan, seed):
        pool = KVPool(B, mb, nb, seed=seed)
        kc = torch.full((nb, Hkv, 64, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
        vc = torch.full_like(kc, float("nan"))
        start, out = [0] * B, [[] for _ in range(B)]
        cap = 400
        for new in plan:
            rows = torch.zeros((cap, d), dtype=torch.bfloat16, device="cuda")
            packed = torch.cat([x[b][start[b]:start[b] + new[b]] for b in range(B)])
            T = len(packed)
            rows[:T] = packed
            pool.resize(i32([s + n for s, n in zip(start, new)]))
            row0, seq, pos = i32([0] * (B + 1)), i32([-1] * cap), i32([-1] * cap)
            slots = torch.full((cap,), -1, dtype=torch.int64, device="cuda")
            bi.bi_slot_map(i32(new), i32(start), B, pool.table, mb, nb, cap, row0, seq, pos, slots)
            q = torch.empty((T, Hq, hd), dtype=torch.bfloat16, device="cuda")
            bi.bi_qkv_rope_kv_write(rows, T, d, w, Hq, Hkv, hd, seq, pos, table, 512, pool.table, mb, nb, q, kc, vc)
            ws = torch.empty(bi.bi_attention_workspace_size(T, Hq, hd, 256, 512), dtype=torch.uint8, device="cuda")
            o = torch.empty((T, Hq * hd), dtype=torch.bfloat16, device="cuda")
            bi.bi_attention(q, T, torch.arange(B, dtype=torch.int32, device="cuda"), row0, i32(start), B, max(new),
                            Hq, Hkv, hd, kc, vc, pool.table, mb, nb, 256, 512, 1 / math.sqrt(hd), ws, o)
            r = row0.cpu().tolist()
            assert r[-1] == T and (slots[T:] == -1).all()
            # the slots are where the projection wrote its rows (NaN before)
            k_at = kc.permute(0, 2, 1, 3).reshape(nb * 64, Hkv, hd)[slots[:T]]
            assert not torch.isnan(k_at.float()).any()
            for b in range(B):
                out[b].append(o[r[b]:r[b + 1]])
            start = [s + n for s, n in zip(start, new)]
        assert bi.bi_device_status() == 0
        return [torch.cat(t) for t in out]

    whole = run([lens], seed=1)
    split = run(steps, seed=2)
    for b in range(B):
        assert same_bits(whole[b], split[b]), b
