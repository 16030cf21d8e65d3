"""The RoPE tables, the rotation and write at slots, the row map and the acceptance of drafted trees, through the
C ABI against the oracle."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from gpu_util import dev_bf16_from_f32, host_f32, same_bits
from oracle import tree
from synthetic import bits_to_f32, to_bf16_bits
from tree_util import i32, make_tree

pytestmark = pytest.mark.gpu

KINDS = {"plain": {}, "linear": dict(factor=4.0), "base": dict(factor=3.0),
         "turns": dict(factor=8.0, orig_len=4096.0, low=1.0, high=4.0),
         "dims": dict(factor=16.0, orig_len=4096.0, low=1.0, high=32.0, amplitude=1.2772588722239782)}


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("max_pos,rot,theta", [(1, 2, 10000.0), (700, 64, 10000.0), (33000, 128, 5e5), (999, 6, 1e4),
                                               (77, 256, 1e6), (20000, 96, 1e4)])
def test_scaled_tables(kind, max_pos, rot, theta):
    if kind == "base" and rot == 2:
        pytest.skip("a scaled base needs rot > 2")
    par = KINDS[kind]
    t = torch.full((max_pos + 1, rot), 9.0, device="cuda")
    bi.bi_rope_scaled_table(t, max_pos, rot, theta, bi.bi_rope_scaling(getattr(bi, "BI_ROPE_" + kind.upper()), **par))
    want = tree.rope_table(max_pos, rot, theta, kind, **par)
    amp = par.get("amplitude", 1.0)
    # 0.6 units in the last place of the amplitude's binade, and the angle's own error on both sides (w <= 1)
    tol = 0.6 * 2.0**-23 * amp + np.arange(max_pos)[:, None] * 2.0**-51 * amp
    assert (np.abs(t[:-1].double().cpu().numpy() - want) <= tol).all()
    assert (t[-1] == 9).all()


def test_plain_table_beside_bi_rope_table_and_one_off_a_boundary():
    a, b = torch.empty((5000, 128), device="cuda"), torch.empty((5000, 128), device="cuda")
    bi.bi_rope_table(a, 5000, 128, 10000.0)
    bi.bi_rope_scaled_table(b, 5000, 128, 10000.0)
    # both within 0.6 units of the exact value
    assert (a - b).abs().max().item() <= 1.2 * 2.0**-23 and (a == b).float().mean().item() > 0.9
    c = torch.empty(5000 * 128 + 1, device="cuda")[1:].view(5000, 128)     # 4-byte aligned
    bi.bi_rope_scaled_table(c, 5000, 128, 10000.0)
    assert same_bits(b, c)


@pytest.mark.parametrize("hq,hkv,hd,rot,inter,pad", [(8, 2, 128, 128, False, 0), (4, 4, 64, 64, True, 8), (3, 1, 80, 16, False, 16),
                                                     (8, 8, 64, 32, False, 0), (2, 1, 96, 24, True, 40), (1, 1, 8, 8, True, 0),
                                                     (2, 2, 64, 0, False, 0), (16, 4, 256, 64, True, 0)])
@pytest.mark.parametrize("T", [1, 37])
def test_rotation_and_write_at_slots(hq, hkv, hd, rot, inter, pad, T):
    rng = np.random.default_rng(hd + T + rot)
    nb, max_pos, ld = 5, 300, (hq + 2 * hkv) * hd + pad
    x = bits_to_f32(to_bf16_bits(rng.normal(size=(T, ld)).astype(np.float32)))
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    slots = rng.permutation(nb * 64)[:T].astype(np.int64)
    table = tree.rope_table(max_pos, max(rot, 2), 1e4).astype(np.float32)
    k = torch.full((nb, hkv, 64, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    v, q = k.clone(), torch.zeros((T, hq, hd), dtype=torch.bfloat16, device="cuda")
    bi.bi_rope_slot_write(dev_bf16_from_f32(x), T, i32(pos), torch.from_numpy(slots).cuda(), hq, hkv, hd,
                          torch.from_numpy(table).cuda(), max_pos, nb, q, k, v, rot=rot,
                          layout=bi.BI_ROPE_INTERLEAVED if inter else bi.BI_ROPE_HALF, ld=ld)
    rows = x[:, :(hq + 2 * hkv) * hd].reshape(T, hq + 2 * hkv, hd)
    cs = table[pos][:, None, :]
    y = tree.rotate(rows[:, :hq + hkv], cs[..., :rot // 2], cs[..., max(rot, 2) // 2:][..., :rot // 2], rot, inter)
    y = bits_to_f32(to_bf16_bits(y))
    wk, wv = np.full((nb, hkv, 64, hd), 5.0, np.float32), np.full((nb, hkv, 64, hd), 5.0, np.float32)
    wk[slots // 64, :, slots % 64], wv[slots // 64, :, slots % 64] = y[:, hq:], rows[:, hq + hkv:]
    assert (host_f32(q) == y[:, :hq]).all() and (host_f32(k) == wk).all() and (host_f32(v) == wv).all()
    assert bi.bi_device_status() == bi.BI_OK


def test_slot_write_has_the_bits_of_rope_kv_write_and_skips_bad_rows():
    T, hq, hkv, hd, nb = 50, 8, 2, 64, 4
    g = torch.Generator("cuda").manual_seed(1)
    qkv = torch.randn((T, (hq + 2 * hkv) * hd), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.empty((400, hd), device="cuda")
    bi.bi_rope_table(table, 400, hd)
    bt = i32([[3, 0, 2]])
    outs = [[torch.zeros((T, hq, hd), dtype=torch.bfloat16, device="cuda")] +
            [torch.zeros((nb, hkv, 64, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    bi.bi_rope_kv_write(qkv, T, i32([0]), i32([0, T]), i32([100]), 1, T, hq, hkv, hd, table, 400, bt, 3, nb, *outs[0])
    pos = np.arange(100, 100 + T)
    slots = np.array([3, 0, 2])[pos // 64] * 64 + pos % 64
    bi.bi_rope_slot_write(qkv, T, i32(pos), torch.from_numpy(slots.astype(np.int64)).cuda(), hq, hkv, hd, table, 400, nb,
                          *outs[1])
    assert all(same_bits(a, b) for a, b in zip(*outs))
    pos[7], slots[9], slots[11] = 400, nb * 64, -1
    q, k, v = [torch.full_like(t, 2.0) for t in outs[0]]
    bi.bi_rope_slot_write(qkv, T, i32(pos), torch.from_numpy(slots.astype(np.int64)).cuda(), hq, hkv, hd, table, 400, nb,
                          q, k, v)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert (q[7] == 2).all() and same_bits(q[[9, 11]], outs[0][0][[9, 11]])
    for i in (7, 9, 11):
        p = 100 + i
        blk = [3, 0, 2][p // 64]
        assert (k[blk, :, p % 64] == 2).all() and (v[blk, :, p % 64] == 2).all()


@pytest.mark.parametrize("B,n", [(1, 1), (3, 5), (8, 31), (9, 32), (40, 33), (300, 64), (17, 256)])
def test_row_map(B, n):
    rng = np.random.default_rng(B * n)
    kinds = ["chain", "levels", "random", "forest"]
    trees = [make_tree(kinds[b % 4], int(rng.integers(0, n + 1)) if b else n, rng) for b in range(B)]
    start = rng.integers(0, 3000, B)
    mb = 60
    table = rng.permutation(B * mb).reshape(B, mb)
    T = sum(len(t) for t in trees)
    counts = [len(t) for t in trees]
    row0 = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    seq, pos = (torch.full((T + 7,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    slot = torch.full((T + 7,), -9, dtype=torch.int64, device="cuda")
    parent = i32(np.concatenate([np.asarray(t, np.int32) for t in trees]))
    bi.bi_tree_slot_map(parent, i32(counts), i32(start), B, n, i32(table), mb, B * mb, T + 7, row0, seq, pos, slot)
    assert bi.bi_device_status() == bi.BI_OK
    want = tree.slot_map(trees, start.tolist(), table.tolist())
    assert row0.cpu().tolist() == np.concatenate([[0], np.cumsum(counts)]).tolist()
    got = list(zip(seq.cpu().tolist(), pos.cpu().tolist(), slot.cpu().tolist()))
    assert got[:T] == want and got[T:] == [(-9, -9, -9)] * 7
    # single outputs
    pos2 = torch.full_like(pos, -9)
    bi.bi_tree_slot_map(parent, i32(counts), i32(start), B, n, None, mb, B * mb, T + 7, row0, None, pos2, None)
    assert torch.equal(pos, pos2)


def test_row_map_faults():
    trees = [[-1, 0, 1], [-1, 1, 0, 1], [-1], [-1, 0]]
    parent = i32(sum(trees, []))
    table = [[0, 1], [2, -1], [3, 4], [9, 5]]

    def call(counts, start, T=10, most=4):
        out = [torch.full((m,), -9, dtype=d, device="cuda") for m, d in
               ((5, torch.int32), (10, torch.int32), (10, torch.int32), (10, torch.int64))]
        bi.bi_tree_slot_map(parent, i32(counts), i32(start), 4, most, i32(table), 2, 8, T, *out)
        return bi.bi_device_status(), [o.cpu().tolist() for o in out]
    st, (row0, seq, pos, slot) = call([3, 4, 1, 2], [63, 62, -1, 60])
    assert st == bi.BI_ERR_DEVICE_CHECK and row0 == [0, 3, 7, 8, 10]
    assert pos == [63, 64, 65, 62, -1, 63, -1, -1, 60, 61]       # node 1 is its own parent, node 3 below it; start -1
    assert slot == [63, 64, 65, 2 * 64 + 62, 2 * 64 + 63, -1, -1, -1, -1, -1]
    st, (row0, seq, pos, slot) = call([3, 4, 1, 2], [0, 0, 0, 0], most=3)
    assert st == bi.BI_ERR_DEVICE_CHECK and seq[3:7] == [-9] * 4 and seq[7:] == [2, 3, 3]
    st, (row0, seq, pos, slot) = call([3, -2, 1, 2], [0, 0, 0, 0], T=5)
    assert st == bi.BI_ERR_DEVICE_CHECK and row0 == [0, 3, 3, 4, 5] and seq == [0, 0, 0, 2] + [-9] * 6


def accept_case(B, n, seed, layers=2, hkv=2, hd=64, agree=0.8):
    rng = np.random.default_rng(seed)
    kinds = ["levels", "chain", "random", "forest"]
    trees = [make_tree(kinds[b % 4], int(rng.integers(0, n + 1)) if b else n, rng) for b in range(B)]
    tokens = [rng.integers(0, 5, len(t)).tolist() for t in trees]          # few tokens: equal siblings
    targets = []
    for t, tok in zip(trees, tokens):
        kids = [[i for i, p in enumerate(t) if p == j] for j in range(len(t))]
        targets.append([tok[kids[j][int(rng.integers(0, len(kids[j])))]] if kids[j] and rng.random() < agree else 99
                        for j in range(len(t))])
    start = rng.integers(0, 150, B)
    mb = (150 + n) // 64 + 2
    nb = B * mb + 1
    table = rng.permutation(nb)[:B * mb].reshape(B, mb)
    k = torch.from_numpy(rng.normal(size=(layers, nb, hkv, 64, hd)).astype(np.float32)).cuda().to(torch.bfloat16)
    return trees, tokens, targets, start, mb, nb, table, k, (k * 3).to(torch.bfloat16)


@pytest.mark.parametrize("B,n,layers,hkv,hd", [(1, 1, 1, 1, 8), (4, 6, 2, 2, 64), (9, 40, 3, 4, 128), (33, 64, 2, 8, 64),
                                               (5, 256, 1, 2, 96)])
@pytest.mark.parametrize("limited", [False, True])
def test_acceptance_and_the_cache(B, n, layers, hkv, hd, limited):
    trees, tokens, targets, start, mb, nb, table, k, v = accept_case(B, n, B + n, layers, hkv, hd)
    rng = np.random.default_rng(1)
    limit = rng.integers(0, 6, B) if limited else np.full(B, 1 << 30)
    most = n if limited else max(1, n // 2)
    row0 = np.concatenate([[0], np.cumsum([len(t) for t in trees])])
    T = int(row0[-1])
    cnt, pos = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    path, out = (torch.full((B, most), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    wk, wv = k.clone(), v.clone()
    bi.bi_tree_accept(i32(sum(trees, [])), i32(row0), i32(start), i32(sum(tokens, [])), i32(sum(targets, [])), B, n, T, most,
                      cnt, path, out, pos, limit=i32(limit) if limited else None, n_layers=layers, Hkv=hkv, hd=hd, k_cache=k,
                      v_cache=v, block_table=i32(table), max_blocks_per_seq=mb, n_blocks=nb)
    assert bi.bi_device_status() == bi.BI_OK
    moved = 0
    for b in range(B):
        p = tree.accept(trees[b], tokens[b], targets[b], min(int(limit[b]), most))
        assert cnt[b].item() == len(p) and pos[b].item() == start[b] + len(p)
        assert path[b].cpu().tolist() == p + [-1] * (most - len(p))
        assert out[b].cpu().tolist() == [targets[b][i] for i in p] + [-1] * (most - len(p))
        at = [(int(table[b, (start[b] + i) // 64]), int(start[b] + i) % 64) for i in range(n)]
        for c in (wk, wv):
            rows = [c[:, at[i][0], :, at[i][1]].clone() for i in p]
            for j, r in enumerate(rows):
                c[:, at[j][0], :, at[j][1]] = r
        moved += sum(i != j for j, i in enumerate(p))
    same = same_bits(k, wk) and same_bits(v, wv)
    assert same and (moved > 0 or n < 40 or B == 1)
    # without caches the same path
    cnt2, path2 = torch.zeros_like(cnt), torch.zeros_like(path)
    bi.bi_tree_accept(i32(sum(trees, [])), i32(row0), i32(start), i32(sum(tokens, [])), i32(sum(targets, [])), B, n, T, most,
                      cnt2, path2, out, pos, limit=i32(limit) if limited else None)
    assert torch.equal(cnt, cnt2) and torch.equal(path, path2)


def test_acceptance_faults():
    # node 0 no root; a child before its parent; rows behind T; a start below zero; a block outside the cache
    trees = [[0, 0], [-1, 2, 1], [-1, 0], [-1, 0], [-1, 0, 0]]
    tokens, targets = [[1, 2]] + [[1, 2, 2]] + [[1, 2]] * 2 + [[1, 5, 2]], [[2, 0], [2, 2, 2], [2, 0], [2, 0], [2, 0, 7]]
    row0 = [0, 2, 5, 7, 9, 13]
    start = [0, 0, 0, -3, 0]
    k = torch.arange(7 * 64, device="cuda").view(1, 7, 1, 64, 1).expand(1, 7, 1, 64, 8).to(torch.bfloat16).contiguous()
    v, keep = k.clone(), k.clone()
    cnt, pos = (torch.full((5,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    path, out = (torch.full((5, 2), -9, dtype=torch.int32, device="cuda") for _ in range(2))

    def call(row0, table):
        bi.bi_tree_accept(i32(sum(trees, [])), i32(row0), i32(start), i32(sum(tokens, [])), i32(sum(targets, [])), 5, 3, 12, 2,
                          cnt, path, out, pos, n_layers=1, Hkv=1, hd=8, k_cache=k, v_cache=v, block_table=i32(table),
                          max_blocks_per_seq=1, n_blocks=7)
        return bi.bi_device_status()
    assert call(row0, [[0], [1], [2], [3], [4]]) == bi.BI_ERR_DEVICE_CHECK
    assert cnt.cpu().tolist() == [0, 1, 2, 0, 0] and same_bits(k, keep)
    assert call(row0[:5] + [12], [[0], [1], [2], [3], [7]]) == bi.BI_ERR_DEVICE_CHECK
    assert cnt.cpu().tolist() == [0, 1, 2, 0, 2] and path[4].cpu().tolist() == [0, 2] and same_bits(k, keep)
    assert call(row0[:5] + [12], [[0], [1], [2], [3], [4]]) == bi.BI_ERR_DEVICE_CHECK
    keep[:, 4, :, 1] = keep[:, 4, :, 2]
    assert same_bits(k, keep) and same_bits(v, keep)
