"""Pools that are not one: what a call leaves of them is told by the device status, and hands no block out twice."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("B", [2, 300])
@pytest.mark.parametrize("free", [3, 4])
def test_blocks_that_do_not_fit_the_ring_are_not_counted(B, free):
    """Four blocks, of which the ring lists `free`, though a request holds two: what it gives back fits as far as
    there are places, and the count is that of the listed ids."""
    table = np.full((B, 4), -1)
    table[0, :2] = [3, 2]
    owned = np.zeros(B)
    owned[0] = 2
    d_table, d_owned, ring, pool = _i32(table), _i32(owned), _i32([0, 1, 2, 3]), _i32([0, free])
    lens = np.zeros(B)
    lens[-1] = 64                                             # one shrinks, one grows
    bi.bi_block_table_resize(_i32(lens), B, d_table, 4, d_owned, ring, 4, pool)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert d_owned.cpu().tolist() == [0] * (B - 1) + [1] and d_table[-1, 0].item() == 0
    assert pool.cpu().tolist() == [1, 3]                      # 3: 2 left and 1 given back; 4: 3 left
    assert ring[1:].cpu().tolist() == [1, 2, 3]               # place 3 takes the first given back, which is 3
    # block 0 is request B - 1's until that gives it back: three are left for the others
    lens[0] = 4 * 64
    bi.bi_block_table_resize(_i32(lens), B, d_table, 4, d_owned, ring, 4, pool)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK and d_owned[0].item() == 0
    lens[0] = 3 * 64
    bi.bi_block_table_resize(_i32(lens), B, d_table, 4, d_owned, ring, 4, pool)
    assert bi.bi_device_status() == 0
    assert d_table[0].cpu().tolist() == [1, 2, 3, -1] and pool.cpu().tolist() == [0, 0]


@pytest.mark.parametrize("B", [2, 300])
@pytest.mark.parametrize("bad", [[-1, 3], [10, 3], [0, 11], [0, -1]])
def test_a_bad_pool_leaves_its_counts_in_other_arrays_too(B, bad):
    """Nothing is changed, so the new counts are the old ones."""
    owned = np.arange(B) % 3
    table = np.full((B, 4), -1)
    d_table, d_owned, ring, pool = _i32(table), _i32(owned), _i32(np.arange(10)), _i32(bad)
    owned_out, pool_out = _i32(np.full(B, -7)), _i32([-7, -7])
    bi.bi_block_table_resize(_i32(np.full(B, 64)), B, d_table, 4, d_owned, ring, 10, pool, n_owned_out=owned_out,
                             pool_out=pool_out)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert owned_out.cpu().tolist() == owned.tolist() == d_owned.cpu().tolist()
    assert pool_out.cpu().tolist() == bad == pool.cpu().tolist()
    assert (d_table == -1).all() and ring.cpu().tolist() == list(range(10))
