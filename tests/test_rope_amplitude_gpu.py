"""The amplitude of a scaled RoPE table is a 64-bit number: the table's bound holds whether or not it is an fp32 one."""
import math

import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from oracle import tree

pytestmark = pytest.mark.gpu

# 0.1 ln(factor) + 1 for factors of 40, 64 and 16; next to one; near a binade's end; large, small and subnormal
AMPLITUDES = [0.1 * math.log(40) + 1, 0.1 * math.log(64) + 1, 0.1 * math.log(16) + 1, 1 + 2.0**-24.01, 1 - 2.0**-25.1,
              1 + 2.0**-40, 1.99999, -math.sqrt(3), 1e38 / 3, 2.0**-100 / 0.75, 1e-42, 0.0]


@pytest.mark.parametrize("amp", AMPLITUDES)
@pytest.mark.parametrize("kind,par", [("plain", {}), ("dims", dict(factor=40.0, orig_len=4096.0, low=1.0, high=32.0))])
@pytest.mark.parametrize("max_pos,rot", [(20000, 64), (333, 6)])
def test_tables_of_any_amplitude(amp, kind, par, max_pos, rot):
    t = torch.full((max_pos, rot), 9.0, device="cuda")
    bi.bi_rope_scaled_table(t, max_pos, rot, 1e4, bi.bi_rope_scaling(getattr(bi, "BI_ROPE_" + kind.upper()), amplitude=amp,
                                                                     **par))
    want = tree.rope_table(max_pos, rot, 1e4, kind, amplitude=amp, **par)
    # In units of 2^-23 |A|.  The larger of sine and cosine of the offset: half a unit (rounding of at most |A|) and 0.05
    # (small terms); the smaller, at most 0.71 |A|: 0.36 and 0.13.  The angle: p w 2^-52 on either side (w <= 1).
    # Subnormal numbers: four roundings of 2^-150.
    tol = abs(amp) * (0.6 * 2.0**-23 + np.arange(max_pos)[:, None] * 2.0**-51) + 2.0**-148
    assert (np.abs(t.double().cpu().numpy() - want) <= tol).all()
