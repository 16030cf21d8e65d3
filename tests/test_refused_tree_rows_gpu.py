"""Sequences that the row map refuses leave no row behind that a step would write to the cache, whatever an earlier step left
in the buffers."""
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from gpu_util import same_bits
from tree_util import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,most,T,refused", [([2, 70, 3], 64, 75, range(2, 72)),      # more nodes than max_nodes
                                                   ([2, 3, 4], 4, 7, range(5, 7)),          # rows behind T
                                                   ([9, 2, 1], 4, 7, range(0, 7)),          # both
                                                   ([2, 2, 1 << 30], 4, 40, range(4, 40))])
def test_rows_of_refused_sequences_write_nothing(counts, most, T, refused):
    rows, hq, hkv, hd, nb, mb = T + 3, 2, 1, 64, 9, 3
    parent = i32([-1] + [0] * (rows - 1))
    for n in range(1, 3):                                  # a root in every sequence
        if sum(counts[:n]) < rows:
            parent[sum(counts[:n])] = -1
    table = i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    row0, seq, pos = i32([-9] * 4), i32([2] * rows), i32([5] * rows)
    slots = torch.full((rows,), 77, dtype=torch.int64, device="cuda")          # an earlier step's
    bi.bi_tree_slot_map(parent, i32(counts), i32([10, 20, 30]), 3, most, table, mb, nb, T, row0, seq, pos, slots)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    for r in range(rows):
        b = next((b for b in range(3) if sum(counts[:b]) <= r < sum(counts[:b + 1])), None)
        got = seq[r].item(), pos[r].item(), slots[r].item()
        if r in refused:
            assert got == (2, -1, -1)
        elif r >= T or b is None:
            assert got == (2, 5, 77)
        else:
            i = r - sum(counts[:b])
            assert got == (b, [10, 20, 30][b] + min(i, 1), b * 192 + [10, 20, 30][b] + i)
    k = torch.full((nb, hkv, 64, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    v, keep = k.clone(), k.clone()
    q = torch.zeros((T, hq, hd), dtype=torch.bfloat16, device="cuda")
    rope = torch.ones((64, hd), device="cuda")
    qkv = torch.randn((T, (hq + 2 * hkv) * hd), device="cuda").to(torch.bfloat16)
    bi.bi_rope_slot_write(qkv, T, pos, slots, hq, hkv, hd, rope, 64, nb, q, k, v)
    bi.bi_device_status()
    written = [s for r, s in enumerate(slots[:T].tolist()) if r not in refused]
    for c in (k, v):
        c = c.clone()
        for s in written:
            assert not same_bits(c[s // 64, :, s % 64], keep[s // 64, :, s % 64])
            c[s // 64, :, s % 64] = 3.0
        assert same_bits(c, keep)
