"""Tokens whose mass is 0 in 64 bits: kept by their place in the order, scored by the formula, never drawn."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from oracle import sampling as osm
from tests.test_sampling_gpu import _f32, _rule, _tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("temp", [1.0, 0.7, 0.013, 3.0])
@pytest.mark.parametrize("top", [0.0, 5.0, -300.0])
def test_the_smallest_mass_that_u_zero_draws(temp, top):
    """Rows of two tokens, the first of which has a mass around 2^-1075, where 64 bits round to 0 or to 2^-1074.
    The oracle's exp is trusted from 4 steps of the logit on, 1e-4 of the mass and more at these sizes."""
    t = _f32(temp)
    edge = float(np.float32(top)) - 745.1332191019411 * t
    x0 = np.float32(edge)
    steps = np.concatenate([np.arange(-40, -3), np.arange(4, 41)])
    first = (x0.astype(np.float64) + steps * float(np.spacing(np.abs(x0)))).astype(np.float32)
    x = np.stack([first, np.full(len(first), top, np.float32)], 1)
    T = len(x)
    dev = torch.from_numpy(x).cuda()
    ids = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((T,), 7.0, device="cuda")
    bi.bi_sample(dev, T, 2, _rule(T, temp=temp), torch.zeros(T, device="cuda"), ids, lp)
    sc = torch.full((T,), 7.0, device="cuda")
    bi.bi_sample_logprob(dev, T, 2, _rule(T, temp=temp), torch.zeros(T, dtype=torch.int32, device="cuda"), sc)
    assert bi.bi_device_status() == 0
    want = [osm.draw(row, 0.0, temperature=t)[0] for row in x]
    assert want == [1 if s < 0 else 0 for s in steps]
    assert ids.cpu().tolist() == want
    for row, got in zip(x, sc.cpu().numpy()):
        w = osm.logprob(row, 0, temperature=t)
        assert abs(float(got) - w) <= _tol(w, w)


@pytest.mark.parametrize("V", [50, 5000, 30001])
@pytest.mark.parametrize("rule", [dict(), dict(k=4), dict(k=1200), dict(p=0.9), dict(mp=0.1)])
def test_tokens_without_mass_are_scored_by_their_place(V, rule):
    """Thousands of scaled logits below the rest: scored when kept, cut in the order, and drawn by no u."""
    rng = np.random.default_rng(V)
    row = (-1500.0 - 10.0 * rng.random(V)).astype(np.float32)
    row[7], row[V // 2] = 3.0, 2.0
    r = dict(top_k=rule.get("k", 0), top_p=_f32(rule.get("p", 1.0)), min_p=_f32(rule.get("mp", 0.0)))
    kept, _ = osm.kept_tokens(row, **r)
    ids = sorted({7, V // 2, int(kept[-1]), int(kept[0]), 0, V - 1, int(np.argmin(row))})
    n = len(ids)
    dev = torch.from_numpy(row).cuda()[None].repeat(n, 1).contiguous()
    lp = torch.full((n,), 7.0, device="cuda")
    bi.bi_sample_logprob(dev, n, V, _rule(n, **rule), torch.tensor(ids, dtype=torch.int32, device="cuda"), lp)
    for i, got in zip(ids, lp.cpu().numpy()):
        want = osm.logprob(row, i, **r)
        assert got == want if np.isinf(want) else abs(float(got) - want) <= _tol(want, want), i
    u = np.array([0.0, 1e-38, 0.3, 0.9, 1 - 2.0 ** -24], np.float32)
    dev = dev[:1].repeat(len(u), 1).contiguous()
    got = torch.full((len(u),), -7, dtype=torch.int32, device="cuda")
    bi.bi_sample(dev, len(u), V, _rule(len(u), **rule), torch.from_numpy(u).cuda(), got)
    assert got.cpu().tolist() == [osm.draw(row, _f32(v), **r)[0] for v in u]
    assert set(got.cpu().tolist()) <= {7, V // 2}
    assert bi.bi_device_status() == 0
