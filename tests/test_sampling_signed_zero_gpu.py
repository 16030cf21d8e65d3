"""u = -0.0 is u = 0: the first kept token, on every way to a draw."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from tests.gpu_util import same_bits
from tests.test_sampling_gpu import RULES, _check, _logits, _rule

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1, 2, 129, 5003, 40001])
@pytest.mark.parametrize("rule", ["greedy", "top1", *RULES])
def test_negative_zero_draws_as_zero(rule, V):
    r = {"greedy": dict(temp=0.0), "top1": dict(k=1)}.get(rule) or RULES[rule]
    rng = np.random.default_rng([V, len(rule)])
    T = 4
    x = _logits(rng, T, V, "peaked")
    dev = torch.from_numpy(x).cuda()
    out = []
    for zero in (-0.0, 0.0):
        u = torch.full((T,), zero, device="cuda")
        ids = torch.full((T,), -7, dtype=torch.int32, device="cuda")
        lp = torch.full((T,), 7.0, device="cuda")
        bi.bi_sample(dev, T, V, _rule(T, **r), u, ids, lp)
        out.append((ids, lp))
    assert torch.equal(out[0][0], out[1][0]) and same_bits(out[0][1], out[1][1])
    _check(x, np.zeros(T), out[0][0].cpu().numpy(), out[0][1].cpu().numpy(), **r)
    assert bi.bi_device_status() == 0
