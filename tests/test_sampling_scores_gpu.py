"""Scores of tokens that were not drawn: the maximum, both sides of each cut, ties on either side of an
index cut, masked and random cut tokens, on every split of a row and on the one-CTA way."""
import math

import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from oracle import sampling as osm
from tests.gpu_util import same_bits
from tests.test_sampling_gpu import RULES, _f32, _logits, _rule, _tol

pytestmark = pytest.mark.gpu

NAMES = dict(temp="temperature", k="top_k", p="top_p", mp="min_p")


def _candidates(x, kept, rng):
    """Tokens whose score tells where the cut is (indices; kept in kept order)."""
    V = len(x)
    inside = np.zeros(V, bool)
    inside[kept] = True
    order = np.lexsort((np.arange(V), -x))
    ids = [int(order[0]), int(kept[-1]), int(kept[len(kept) // 2])]
    n = len(kept)
    ids.append(int(order[n]) if n < V else int(order[-1]))                     # the first cut token
    same = np.flatnonzero(x == x[kept[-1]])                                    # ties of the last kept value
    ids += [int(same[0]), int(same[-1])]
    cut = np.flatnonzero(~inside)
    ids.append(int(rng.choice(cut)) if len(cut) else 0)
    low = np.flatnonzero(x == -np.inf)
    ids.append(int(low[0]) if len(low) else int(order[-1]))
    ids.append(int(rng.integers(0, V)))
    return ids


def _row(dist, rng, V):
    if dist == "far":       # beyond 2^13 octaves above zero: the masses' other form
        x = (3e4 + 30.0 * rng.standard_normal(V)).astype(np.float32)
        x[rng.integers(0, V, V // 10)] = np.float32(3e4)
        return x
    x = _logits(rng, 1, V, dist)[0]
    x[rng.integers(1, V, 5)] = -np.inf
    return x


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("dist", ["flat", "peaked", "coarse", "wide", "far"])
@pytest.mark.parametrize("V,dtype", [(20001, torch.float32), (20001, torch.bfloat16), (300, torch.float32)])
def test_scores_around_every_cut(rule, dist, V, dtype):
    rng = np.random.default_rng([V, len(rule), len(dist), 5])
    r = {NAMES[k]: v if k == "k" else _f32(v) for k, v in RULES[rule].items()}
    rows, ids, want, z = [], [], [], []
    for j in range(4):
        x = torch.from_numpy(_row(dist, rng, V)).to(dtype).float().numpy()
        kept, zz = osm.kept_tokens(x, **r)
        total = math.log(math.fsum(np.exp(zz[kept])))
        inside = set(kept.tolist())
        for i in _candidates(x, kept, rng):
            rows.append(x)
            ids.append(i)
            want.append(zz[i] - total if i in inside else -np.inf)
            z.append(zz[i])
        assert want[-9] == osm.logprob(x, ids[-9], **r)
    n = len(ids)                                           # 36 rows: 8 CTAs a row; 72: 4; 144: 2; 324: 1
    kind = bi.BI_DTYPE_BF16 if dtype == torch.bfloat16 else bi.BI_DTYPE_FP32
    dev = torch.from_numpy(np.stack(rows)).cuda().to(dtype)
    d_ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
    first = None
    for times in (1, 2, 4, 9):
        T = n * times
        lp = torch.full((T,), 7.0, device="cuda")
        bi.bi_sample_logprob(dev.repeat(times, 1), T, V, _rule(T, **RULES[rule]), d_ids.repeat(times), lp, dtype=kind)
        first = lp[:n] if first is None else first
        assert same_bits(lp, first.repeat(times)), times
    assert bi.bi_device_status() == 0
    for t, got in enumerate(first.cpu().numpy()):
        if want[t] == -np.inf:
            assert got == -np.inf, (t, ids[t], got)
        else:
            assert abs(float(got) - want[t]) <= _tol(z[t], want[t]), (t, ids[t], got, want[t])
