"""bi_block_table_resize and bi_slot_map on the GPU through the C ABI, exactly the oracle's, and one
step planned by them through the QKV projection and attention."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from oracle import paging

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Pool:
    """The oracle's state beside the device's."""

    def __init__(self, B, mb, nb, seed, head=0):
        self.B, self.mb, self.nb = B, mb, nb
        ids = np.random.default_rng(seed).permutation(nb)
        self.table, self.owned, self.free = [[-1] * mb for _ in range(B)], [0] * B, [int(i) for i in ids]
        self.d_table = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
        self.d_owned = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.d_ring = _i32(np.roll(ids, head))
        self.d_pool = _i32([head, nb])

    def step(self, lens, extra=0, expect_failed=None):
        self.table, self.owned, self.free, failed = paging.resize([int(n) for n in lens], extra, self.table,
                                                                  self.owned, self.free)
        bi.bi_block_table_resize(_i32(lens), self.B, self.d_table, self.mb, self.d_owned, self.d_ring, self.nb,
                                 self.d_pool, extra=extra)
        st = bi.bi_device_status()
        assert st == (bi.BI_ERR_DEVICE_CHECK if failed else bi.BI_OK)
        self.same()
        return failed

    def same(self):
        assert self.d_table.cpu().tolist() == self.table
        assert self.d_owned.cpu().tolist() == self.owned
        head, count = self.d_pool.cpu().tolist()
        ring = self.d_ring.cpu().numpy()
        assert ring[(head + np.arange(count)) % self.nb].tolist() == self.free


@pytest.mark.parametrize("B,mb,nb", [(1, 1, 1), (3, 2, 4), (33, 9, 200), (64, 64, 4096), (64, 70, 3000),
                                     (1025, 5, 4000), (5000, 12, 40000)])
def test_tables_follow_the_oracle_over_many_steps(B, mb, nb):
    rng = np.random.default_rng(B + nb)
    pool = Pool(B, mb, nb, seed=B, head=nb // 3)
    lens = np.zeros(B, np.int64)
    for k in range(6):
        kind = rng.random(B)
        lens = np.where(kind < 0.25, 0, np.where(kind < 0.6, lens + rng.integers(0, 70, B),
                                                 rng.integers(0, mb * 64 + 1, B)))
        lens = np.minimum(lens, mb * 64 - 1)
        pool.step(lens, extra=k % 2)


def test_shortage_is_served_in_request_order():
    pool = Pool(6, 8, 10, seed=3)
    # 4 + 3 blocks, then 4 (short), then 1: it fails too, since the failed request's demand stays counted
    assert pool.step([256, 192, 256, 64, 0, 0]) == [2, 3]
    assert pool.step([256, 0, 256, 64, 0, 0]) == [2, 3]      # what request 1 gives back serves later calls
    assert pool.step([256, 0, 256, 64, 0, 0]) == []
    assert pool.step([256, 0, 256, 64, 0, 9 * 64]) == [5]    # more than the table's columns


def test_out_of_place_leaves_the_counts():
    pool = Pool(64, 80, 3000, seed=5)
    lens = np.random.default_rng(5).integers(1, 2000, 64)
    owned, cnt = torch.zeros_like(pool.d_owned), torch.zeros_like(pool.d_pool)
    before = pool.d_pool.clone()
    for _ in range(2):                                       # the same call twice: the same result
        bi.bi_block_table_resize(_i32(lens), 64, pool.d_table, 80, pool.d_owned, pool.d_ring, 3000, pool.d_pool,
                                 n_owned_out=owned, pool_out=cnt)
        assert pool.d_owned.sum().item() == 0 and torch.equal(pool.d_pool, before)
        assert owned.cpu().tolist() == [-(-int(n) // 64) for n in lens]
        assert cnt[1].item() == 3000 - int(owned.sum())
    assert bi.bi_device_status() == 0


def test_bad_pool_changes_nothing():
    for bad in ([-1, 3], [10, 3], [0, 11], [0, -1]):
        pool = Pool(2, 4, 10, seed=1)
        pool.d_pool.copy_(_i32(bad))
        bi.bi_block_table_resize(_i32([64, 64]), 2, pool.d_table, 4, pool.d_owned, pool.d_ring, 10, pool.d_pool)
        assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
        assert (pool.d_table == -1).all() and pool.d_owned.sum().item() == 0 and pool.d_pool.cpu().tolist() == bad


def test_a_captured_decode_step_grows_its_tables():
    """One graph: resize, then advance the positions; replayed over two block borders."""
    pool = Pool(3, 6, 18, seed=7)
    lens = np.array([60, 1, 130])
    pool.step(lens)
    pos = _i32(lens)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    args = (pos, 3, pool.d_table, 6, pool.d_owned, pool.d_ring, 18, pool.d_pool)
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            bi.bi_block_table_resize(*args, extra=1)
            pos.add_(1)
        for _ in range(80):
            g.replay()
        st.synchronize()
    for k in range(80):
        pool.table, pool.owned, pool.free, _ = paging.resize([int(n) + k for n in lens], 1, pool.table, pool.owned,
                                                             pool.free)
    pool.same()


@pytest.mark.parametrize("B,most,T_extra", [(1, 1, 0), (1, 5000, 3), (64, 1, 0), (200, 90, 77), (700, 3, 1),
                                            (6, 3000, -100)])
def test_slot_map_matches_the_oracle(B, most, T_extra):
    rng = np.random.default_rng(B + most)
    mb = -(-(most + 500) // 64)
    new = rng.integers(0, most + 1, B)
    new[0] = most
    if B > 8:
        new[rng.random(B) < 0.3] = 0                         # empty requests, some at the end
        new[-2:] = 0
    start = rng.integers(0, 400, B)
    table = rng.permutation(B * mb).reshape(B, mb)
    rows = int(new.sum())
    T = max(1, rows + T_extra)
    row0 = torch.full((B + 1,), -5, dtype=torch.int32, device="cuda")
    seq = torch.full((T,), -5, dtype=torch.int32, device="cuda")
    pos = torch.full((T,), -5, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -5, dtype=torch.int64, device="cuda")
    bi.bi_slot_map(_i32(new), _i32(start), B, _i32(table), mb, B * mb, T, row0, seq, pos, slots)
    want0, want = paging.slot_map(new.tolist(), start.tolist(), table.tolist(), T)
    assert bi.bi_device_status() == (bi.BI_ERR_DEVICE_CHECK if rows > T else 0)
    assert row0.cpu().tolist() == want0
    n = len(want)
    got = list(zip(seq.cpu().tolist(), pos.cpu().tolist(), slots.cpu().tolist()))
    assert got[:n] == want
    assert got[n:] == [(-5, -5, -5)] * (T - n)               # rows behind the last sequence are left


def test_slot_map_reports_positions_without_a_block():
    row0 = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    tab = _i32([[3, -1], [99, 1]])
    bi.bi_slot_map(_i32([3, 3]), _i32([63, 126]), 2, tab, 2, 10, 6, row0, slots=slots)
    assert slots.cpu().tolist() == [3 * 64 + 63, -1, -1, 64 + 62, 64 + 63, -1]
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK


def test_slots_pass_32_bits():
    nb = 1 << 26
    row0 = torch.zeros(2, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    bi.bi_slot_map(_i32([2]), _i32([62]), 1, _i32([[nb - 1]]), 1, nb, 2, row0, slots=slots)
    assert slots.cpu().tolist() == [(nb - 1) * 64 + 62, (nb - 1) * 64 + 63]
    assert bi.bi_device_status() == 0


def test_bad_ids_are_moved_and_reported():
    """The resize indexes nothing by a block id, so it only passes a bad one on, with the device status set."""
    for bad in (-1, 10, 1 << 30):
        pool = Pool(2, 4, 10, seed=1)
        pool.d_ring[1] = bad
        bi.bi_block_table_resize(_i32([64, 128]), 2, pool.d_table, 4, pool.d_owned, pool.d_ring, 10, pool.d_pool)
        assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
        assert pool.d_owned.cpu().tolist() == [1, 2] and pool.d_table[1, 0].item() == bad
        bi.bi_block_table_resize(_i32([64, 0]), 2, pool.d_table, 4, pool.d_owned, pool.d_ring, 10, pool.d_pool)
        assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
        assert pool.d_owned.cpu().tolist() == [1, 0] and pool.d_pool.cpu().tolist() == [3, 9]


def test_positions_past_31_bits_are_reported():
    row0 = torch.zeros(2, dtype=torch.int32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    bi.bi_slot_map(_i32([3]), _i32([2 ** 31 - 3]), 1, None, 1, 1, 3, row0, row_pos=pos)
    assert pos.cpu().tolist() == [2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1] and bi.bi_device_status() == 0
    for start in (2 ** 31 - 2, -1):
        bi.bi_slot_map(_i32([3]), _i32([start]), 1, None, 1, 1, 3, row0, row_pos=pos)
        assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
