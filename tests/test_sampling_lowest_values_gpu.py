"""Scores of tokens so far below the row's maximum that (x - max) / T leaves fp32: -inf, the rounding of
the exact value, and the formula's finite value where it stays inside."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from oracle import sampling as osm
from tests.test_sampling_gpu import _f32, _rule, _tol

pytestmark = pytest.mark.gpu

LOWEST = {torch.float32: float(torch.finfo(torch.float32).min), torch.bfloat16: float(torch.finfo(torch.bfloat16).min)}


def _score(row, ids, dtype, **rule):
    """Scores of several tokens of one row, and the oracle's, rounded to fp32."""
    n, V = len(ids), len(row)
    dev = torch.from_numpy(row).to("cuda", dtype)[None].repeat(n, 1).contiguous()
    lp = torch.full((n,), 7.0, device="cuda")
    kind = bi.BI_DTYPE_BF16 if dtype == torch.bfloat16 else bi.BI_DTYPE_FP32
    bi.bi_sample_logprob(dev, n, V, _rule(n, **rule), torch.tensor(ids, dtype=torch.int32, device="cuda"), lp,
                         dtype=kind)
    assert bi.bi_device_status() == 0
    x = dev[0].float().cpu().numpy()
    names = dict(temp="temperature", k="top_k", p="top_p", mp="min_p")
    r = {names[k]: _f32(v) if k != "k" else v for k, v in rule.items()}
    want = np.array([osm.logprob(x, i, **r) for i in ids])
    z = (x[ids].astype(np.float64) - x.max()) / (r.get("temperature") or 1.0)
    return lp.cpu().numpy(), want, z


def _same(got, want, z):
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    for g, w, w32, zz in zip(got, want, want32, z):
        if np.isinf(w32):
            assert g == w32, (g, w)
        else:
            assert abs(float(g) - w) <= _tol(zz, w), (g, w)


@pytest.mark.parametrize("V", [40, 6000, 40001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_by_the_lowest_value(V, dtype):
    """Ten tokens are left, the others hold the type's lowest value: every kind of token is scored."""
    rng = np.random.default_rng(V)
    row = np.full(V, LOWEST[dtype], np.float32)
    left = np.sort(rng.choice(V, 10, replace=False))
    row[left] = rng.uniform(1.0, 10.0, 10)
    masked = np.setdiff1d(np.arange(V), left)
    ids = [int(left[0]), int(left[-1]), int(masked[0]), int(masked[9]), int(masked[10]), int(masked[-1])]
    for temp in (0.5, 0.7, 1.0, 1.5, 1e-3):
        # the whole row, and a top-k that reaches ten masked tokens, 15 and all but one of them
        for k in (0, 20, 25, V - 1):
            _same(*_score(row, ids, dtype, temp=temp, k=k))
    _same(*_score(row, ids, dtype, temp=0.7, p=0.999))
    _same(*_score(row, ids, dtype, temp=0.7, mp=1e-30))


@pytest.mark.parametrize("V", [8, 9000])
def test_differences_beyond_fp32(V):
    """x - max itself overflows, and stays just inside."""
    row = np.full(V, -3e38, np.float32)
    row[1] = 3e38
    row[3] = 2.0
    row[5] = np.finfo(np.float32).min
    ids = [0, 1, 3, 5, V - 1]
    for temp in (0.5, 1.0, 1.7, 2.0, 1e6):
        for rule in (dict(), dict(k=3), dict(k=V - 1), dict(mp=0.5)):
            _same(*_score(row, ids, torch.float32, temp=temp, **rule))


def test_the_borders_of_fp32_at_a_small_temperature():
    """Scores either side of fp32's range: -FLT_MAX / 2^-20 and what is 2^-20 of it."""
    row = np.array([0.0, np.finfo(np.float32).min, -3.2e32, -3.3e32, -1e32, -1.0], np.float32)
    _same(*_score(row, list(range(6)), torch.float32, temp=2.0 ** -20))
    _same(*_score(row, list(range(6)), torch.float32, temp=2.0 ** -64))
