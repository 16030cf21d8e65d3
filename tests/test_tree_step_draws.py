"""A drafted step takes its uniforms as a tensor or from a function: either is checked before the step writes to the cache
(the calls of the library are recorded, nothing is launched)."""
import types

import pytest
import torch

from invariant_forward_policy_gb300 import _lib, decoder
from invariant_forward_policy_gb300.decoder import Decoder, KVCache
from synthetic import DecoderShape

T, B = 6, 2


@pytest.fixture
def step(monkeypatch):
    calls = []

    def record(name):
        def call(*args, **kw):
            calls.append((name, args))
            return 64 if name.endswith("_size") else None
        return call
    monkeypatch.setattr(decoder, "L", types.SimpleNamespace(
        **{n: record(n) if n in _lib.EXPORTED else getattr(_lib, n) for n in dir(_lib) if n.startswith(("bi_", "BI_"))}))
    dec = object.__new__(Decoder)
    dec.shape, dec.device, dec.fp8, dec.max_pos = DecoderShape(1, 128, 4, 2, 64, 256, 512), torch.device("cpu"), False, 128
    dec.w = dict(embed=None, lm_head=None, final_norm=None)
    dec.layers = [{k: torch.zeros((256, 128)) for k in ("attn_norm", "wqkv", "wo", "ffn_norm", "w13", "w2")}]
    dec.rope_table = None
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)

    def run(u):
        calls.clear()
        dec.tree_step(i32(*range(T)), i32(-1, 0, 0, -1, 0, 1), i32(3, 3), i32(5, 9), 4, KVCache([None], [None], 4),
                      torch.zeros((B, 2), dtype=torch.int32), 64, sampling=object(), u=u)
        return calls
    run.calls = calls
    return run


GOOD = torch.rand(T)
BAD = [torch.rand(T, dtype=torch.float64), torch.rand(T - 1), torch.rand(T + 1), torch.rand(2 * T)[::2], torch.rand(T).numpy(),
       torch.empty(T, device="meta"), None]


@pytest.mark.parametrize("u", BAD[:6])
def test_a_tensor_that_is_no_row_of_draws_is_refused(step, u):
    with pytest.raises(ValueError, match="fp32"):
        step(u)
    assert not step.calls


@pytest.mark.parametrize("u", BAD)
def test_a_function_that_gives_no_row_of_draws_is_refused(step, u):
    with pytest.raises(ValueError, match="fp32"):
        step(lambda seq, pos: u)
    assert "bi_rope_slot_write" not in [n for n, _ in step.calls]


@pytest.mark.parametrize("u", [GOOD, GOOD.view(T, 1), lambda seq, pos: GOOD])
def test_draws_reach_the_sampler(step, u):
    (args,) = [a for n, a in step(u) if n == "bi_sample"]
    assert any(isinstance(a, torch.Tensor) and a.data_ptr() == GOOD.data_ptr() for a in args)
