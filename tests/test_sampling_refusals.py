"""Refusals of the sampling and paged-cache planning entry points: every bad argument is answered on the
host before anything is launched (dummy addresses; no GPU is reached)."""
import ctypes

import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300 import _lib
from invariant_forward_policy_gb300.decoder import Decoder, KVCache, KVPool

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="passes dummy addresses: a regressed check must not be able to launch")
INVALID, SHAPE = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _params(n, **arrays):
    s = bi.bi_sampling()
    for name, addr in arrays.items():
        setattr(s, name, addr)
    s.n = n
    return ctypes.byref(s)


def test_sample(lib):
    def call(logits=16, dtype=1, T=4, V=100, ld=100, sp=None, prow=None, u=16, u_rows=1, u_row=None, ids=16, lp=16):
        return lib.bi_sample(logits, dtype, T, V, ld, sp, prow, u, u_rows, u_row, ids, lp, None)
    assert call(T=0, logits=None, u=None, ids=None) == bi.BI_OK
    assert call(T=-1) == INVALID
    assert call(logits=None) == INVALID and "null" in bi.bi_last_error()
    assert call(u=None) == INVALID and call(ids=None) == INVALID
    assert call(dtype=2) == INVALID and "dtype" in bi.bi_last_error()
    assert call(V=0, ld=0) == INVALID and call(ld=99) == INVALID
    assert call(V=262145, ld=262145) == SHAPE
    assert call(u_rows=0) == INVALID
    assert call(T=1 << 31) == INVALID and call(ld=1 << 41) == INVALID
    assert call(logits=18) == INVALID and call(logits=17, dtype=0) == INVALID      # not aligned to the type
    assert call(sp=_params(3, top_p=16)) == INVALID                                # fewer entries than rows
    assert call(sp=_params(0, top_k=16), prow=16) == INVALID


def test_sample_logprob(lib):
    def call(logits=16, dtype=0, T=4, V=100, ld=100, sp=None, prow=None, ids=16, lp=16):
        return lib.bi_sample_logprob(logits, dtype, T, V, ld, sp, prow, ids, lp, None)
    assert call(T=0, logits=None, ids=None, lp=None) == bi.BI_OK
    assert call(T=-5) == INVALID
    for bad in (dict(logits=None), dict(ids=None), dict(lp=None), dict(dtype=-1), dict(V=-1), dict(ld=5),
                dict(logits=3), dict(sp=_params(2, min_p=16))):
        assert call(**bad) == INVALID, bad
    assert call(V=300000, ld=300000) == SHAPE


def test_block_table_resize(lib):
    def call(lens=64, extra=0, B=4, table=64, mb=8, owned=1024, ring=64, nb=10, pool=64, owned_out=4096, pool_out=64):
        return lib.bi_block_table_resize(lens, extra, B, table, mb, owned, ring, nb, pool, owned_out, pool_out, None)
    assert call(B=0, lens=None, table=None) == bi.BI_OK
    for name in ("lens", "table", "owned", "ring", "pool", "owned_out", "pool_out"):
        assert call(**{name: None}) == INVALID, name
    assert call(B=-1) == INVALID and call(mb=0) == INVALID and call(nb=0) == INVALID
    assert call(extra=-1) == INVALID and call(extra=1 << 31) == INVALID
    assert call(B=1 << 20, mb=1 << 12) == INVALID                                  # table beyond 2^31 entries
    assert call(owned=1024, owned_out=1028) == INVALID                             # overlapping, not the same


def test_slot_map(lib):
    def call(new=16, start=16, B=4, table=16, mb=8, nb=10, T=100, row0=16, seq=16, pos=16, slots=16):
        return lib.bi_slot_map(new, start, B, table, mb, nb, T, row0, seq, pos, slots, None)
    assert call(B=0, new=None) == bi.BI_OK
    for bad in (dict(B=-1), dict(T=-1), dict(new=None), dict(start=None), dict(row0=None), dict(table=None),
                dict(mb=0), dict(nb=0), dict(T=1 << 31)):
        assert call(**bad) == INVALID, bad


def test_sampling_structure():
    f, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="fp32"):
        bi.bi_sampling(temperature=i)
    with pytest.raises(ValueError, match="fp32"):
        bi.bi_sampling(top_k=f)
    with pytest.raises(ValueError, match="GPU"):
        bi.bi_sampling(temperature=f)
    with pytest.raises(ValueError, match="contiguous"):
        bi.bi_sampling(top_p=torch.zeros(8)[::2])
    assert bi.bi_sampling().n == 0


def test_sampling_forward_refusals(lib):
    cu = (ctypes.c_int64 * 2)(0, 4)
    # no model, no random numbers or targets, both of them: refused before the model is looked at twice
    assert lib.bi_forward_decode_sample(None, 16, 16, 1, None, 16, 1, None, 16, 1, 16, 16, 1, 64, 16, 16, 16, 1 << 20,
                                        0, None) == INVALID
    args = [cu, cu, None, 1, 64, 16, 1, 16, 16, 1, 16, 16, 16, 1 << 20, 64, 64, 64, 0, None]
    assert lib.bi_forward_prefill_sample(None, 16, 16, None, None, *args) == INVALID
    assert lib.bi_forward_sample_workspace_size(None, 1, 1, 1, 1, 0) == 0
    cfg = _lib.bi_model_config(n_layers=2, d=128, n_heads_q=4, n_heads_kv=2, head_dim=64, ffn=256, vocab=512, eps=1e-6,
                               rope_theta=1e4, kv_block=64, kv_split=512, max_pos=256)
    plain = _lib.bi_forward_workspace_size(cfg, 64, 4, 128, 32)
    assert _lib.bi_forward_sample_workspace_size(cfg, 64, 4, 128, 32) >= plain + 32 * 512 * 4


def test_planning_sizes(lib):
    """Sizes whose index arithmetic would leave 32 bits."""
    assert lib.bi_block_table_resize(64, 0, (1 << 30) + 1, 64, 1, 1 << 40, 64, 10, 64, 1 << 40, 64, None) == INVALID
    assert lib.bi_slot_map(16, 16, (1 << 30) + 1, 16, 8, 10, 100, 16, 16, 16, 16, None) == INVALID


def test_pool_and_decoder_arguments():
    """The decoder's own checks, before anything reaches the device."""
    for sizes in ((0, 4, 4), (4, 0, 4), (4, 4, 0)):
        with pytest.raises(ValueError, match="positive"):
            KVPool(*sizes, device="cpu")
    pool = KVPool(3, 4, 12, device="cpu")
    for lens in (torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(3),
                 torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="lens"):
            pool.resize(lens)
    dec = object.__new__(Decoder)
    dec.device = "cpu"
    cache = KVCache(None, None, 12)
    prompts = [[1, 2], [3], [4, 5, 6]]
    rules, u = bi.bi_sampling(), torch.zeros(5, 3)
    with pytest.raises(ValueError, match="together"):
        dec.rollout(prompts, 5, cache, None, sampling=rules)
    for bad in (torch.zeros(3, 5), torch.zeros(5, 3, dtype=torch.float64), torch.zeros(3, 5).T):
        with pytest.raises(ValueError, match="uniforms"):
            dec.rollout(prompts, 5, cache, None, sampling=rules, uniforms=bad)
    for bad in (KVPool(2, 4, 12, device="cpu"), KVPool(3, 4, 13, device="cpu")):  # sequences, blocks beyond the cache
        with pytest.raises(ValueError, match="pool"):
            dec.rollout(prompts, 5, cache, None, sampling=rules, uniforms=u, pool=bad)
    with pytest.raises(ValueError, match="without sampling"):
        dec.prefill(prompts, cache, None, u=torch.zeros(6))
    with pytest.raises(ValueError, match="either"):
        dec.prefill(prompts, cache, None, sampling=rules)
    with pytest.raises(ValueError, match="either"):
        dec.prefill(prompts, cache, None, sampling=rules, u=torch.zeros(6), targets=prompts)
    for bad in (torch.zeros(5), torch.zeros(6, dtype=torch.float64), torch.zeros(12)[::2]):
        with pytest.raises(ValueError, match="u must"):
            dec.prefill(prompts, cache, None, sampling=rules, u=bad)
    few = bi.bi_sampling()
    few.tensors, few.n = (torch.ones(2), None, None, None), 2
    with pytest.raises(ValueError, match="fewer"):
        dec.recompute(prompts, [[1], [2], [3]], cache, None, sampling=few)
