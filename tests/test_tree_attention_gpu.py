"""bi_tree_attention through the C ABI: bit for bit bi_attention on each node's own path, against the 64-bit
oracle, and the calls at the edges of its contract."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from gpu_util import dev_bf16_from_f32, host_f32, same_bits
from oracle import tree
from tree_util import Case, i32, make_tree

pytestmark = pytest.mark.gpu

HEADS = [(8, 8, 64), (4, 2, 64), (16, 1, 64), (32, 1, 64), (2, 2, 128), (8, 2, 128), (8, 1, 128), (16, 1, 128)]


@pytest.mark.parametrize("hq,hkv,hd", HEADS)
@pytest.mark.parametrize("kind,n", [("chain", 1), ("chain", 3), ("levels", 7), ("random", 16), ("forest", 33)])
def test_rows_are_plain_decode_rows_bitwise(hq, hkv, hd, kind, n):
    rng = np.random.default_rng(n + hd + hq)
    starts = [0, 1, 15, 63, 64, 70, 127, 200, 509]
    trees = [make_tree(kind, n, rng) for _ in starts]
    c = Case(trees, starts, hq, hkv, hd, seed=n)
    assert same_bits(c.run(), c.linear())
    assert bi.bi_device_status() == bi.BI_OK


@pytest.mark.parametrize("hq,hkv,hd,kind,n", [(8, 2, 128, "chain", 90), (2, 2, 64, "chain", 200), (8, 2, 128, "levels", 64),
                                              (4, 4, 64, "levels", 129), (4, 1, 128, "random", 256)])
def test_long_trees_across_lanes_and_splits(hq, hkv, hd, kind, n):
    rng = np.random.default_rng(n)
    starts = [500, 1023, 64, 3]
    c = Case([make_tree(kind, n, rng) for _ in starts], starts, hq, hkv, hd, seed=n + 1)
    assert same_bits(c.run(), c.linear())


@pytest.mark.parametrize("split", [64, 128, 192, 320, 512, 1024, 2048])
@pytest.mark.parametrize("n", [2, 6, 24])
def test_every_split_size(split, n):
    rng = np.random.default_rng(split)
    starts = [0, 60, 333, 1400, 2047]
    c = Case([make_tree("levels", n, rng) for _ in starts], starts, 8, 2, 128, seed=split)
    assert same_bits(c.run(split=split), c.linear(split=split))


@pytest.mark.parametrize("B,most,hq,hkv,hd,n", [(300, 900, 4, 2, 64, 3), (24, 3500, 8, 2, 128, 9), (3, 9000, 16, 4, 128, 40)])
def test_many_and_long_sequences(B, most, hq, hkv, hd, n):
    """More sequences than threads of a CTA, runs of units over several row tiles and sequences, empty ones among them."""
    rng = np.random.default_rng(B)
    starts = [int(s) for s in rng.integers(0, most, B)]
    trees = [make_tree(("levels", "chain", "forest")[b % 3], 0 if b % 7 == 3 else int(rng.integers(1, n + 1)), rng)
             for b in range(B)]
    trees[0] = make_tree("levels", n, rng)
    c = Case(trees, starts, hq, hkv, hd, seed=B, qscale=2.0)
    assert same_bits(c.run(), c.linear())
    assert bi.bi_device_status() == bi.BI_OK


@pytest.mark.parametrize("hq,hkv,hd,n,qscale", [(8, 8, 64, 16, 1.0), (16, 4, 128, 12, 3.0), (8, 2, 128, 33, 1.0)])
def test_against_the_oracle(hq, hkv, hd, n, qscale):
    rng = np.random.default_rng(3)
    starts = [0, 40, 700]
    trees = [make_tree("levels", n, rng), make_tree("chain", n, rng), make_tree("forest", n, rng)]
    c = Case(trees, starts, hq, hkv, hd, seed=9, qscale=qscale)
    got = host_f32(c.run()).reshape(c.T, hq, hd)
    for b, t in enumerate(trees):
        r0 = c.row0[b]
        q = c.q[r0:r0 + n]
        want, spread = tree.attention(q, c.k[b], c.v[b], t, starts[b], c.scale)
        # weights: bf16 P (2^-8), the fp32 scores' sums (hd roundings of the sum of |q k|, in numerator and denominator)
        # and fp32 sums over keys; the output's own rounding (2^-8)
        size = np.abs(q).max(axis=(0, 2)).max() * np.abs(c.k[b]).max() * hd * c.scale
        rel = 2.0**-8 + 2 * hd * 2.0**-24 * size + (starts[b] + n) * 2.0**-24 + 1e-6
        assert (np.abs(got[r0:r0 + n] - want) <= rel * spread + 2.0**-8 * np.abs(want) + 1e-30).all()


def test_rows_do_not_depend_on_the_batch_or_the_other_nodes():
    rng = np.random.default_rng(5)
    trees = [make_tree("random", n, rng) for n in (20, 1, 0, 9)]
    starts = [300, 77, 10, 0]
    c = Case(trees, starts, 8, 2, 128, seed=2)
    whole = c.run()
    for b in (0, 1, 3):
        one = Case([trees[b]], [starts[b]], 8, 2, 128, seed=2)
        one.k, one.v, one.q = [c.k[b]], [c.v[b]], c.q[c.row0[b]:c.row0[b + 1]]
        assert same_bits(one.run(), whole[c.row0[b]:c.row0[b + 1]])
    # nodes off a path do not matter, whatever they hold
    t = trees[0]
    p = tree.path(t, 19)
    for j in range(20):
        if j not in p:
            c.k[0][300 + j] = np.nan
            c.v[0][300 + j] = np.inf
    assert same_bits(c.run()[19], whole[19])


def test_infinite_and_nan_values_on_a_path_stay_on_it():
    t = [-1, 0, 0, 1, 2]
    c = Case([t, [-1, 0]], [70, 20], 4, 2, 64, seed=4)
    plain = c.run()
    c.v[0][71] = np.inf          # node 1: seen by nodes 1 and 3
    c.k[0][72] = np.nan          # node 2: seen by nodes 2 and 4
    got, want = c.run(), c.linear()
    assert same_bits(got[[0, 5, 6]], plain[[0, 5, 6]])
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    assert torch.isnan(got[[2, 4]]).all() and not torch.isfinite(got[[1, 3]]).any()


def test_scores_of_minus_infinity():
    c = Case([[-1, 0]], [130], 2, 2, 64, seed=4)
    c.k[0][:66] = -np.inf        # a first tile (and part of the next) that no row can see
    c.q[:] = np.abs(c.q) + 0.1
    assert same_bits(c.run(), c.linear()) and torch.isfinite(c.run()).all()


def test_rows_behind_the_last_sequence_stay():
    c = Case([make_tree("levels", 6, np.random.default_rng(1))] * 2, [65, 3], 8, 8, 64, seed=1, extra_rows=5)
    out = torch.full((c.T + 5, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out, T=c.T + 5)
    assert (out[c.T:] == 3).all() and same_bits(out[:c.T], c.linear())


def test_faulty_trees_give_zeros_and_the_status():
    rng = np.random.default_rng(0)
    trees = [make_tree("levels", 8, rng) for _ in range(4)]
    c = Case(trees, [100, 130, 510, 9], 8, 2, 128, seed=6)
    good = c.run()
    assert bi.bi_device_status() == bi.BI_OK
    p = np.concatenate(trees).astype(np.int32)
    bad = p.copy()
    bad[8 + 3] = 3               # sequence 1, node 3: its own parent
    bad[16 + 2] = -2             # sequence 2, node 2
    out = c.run(parent=i32(bad))
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    for b in range(4):
        for i in range(8):
            row = out[b * 8 + i]
            if tree.path(list(bad[b * 8:b * 8 + 8]), i) is None:
                assert (row == 0).all()
            else:
                assert same_bits(row, good[b * 8 + i])
    # a start below zero, one whose nodes leave the block table, a position behind max_ctx's last split
    for start, zero in (([-1, 130, 510, 9], 0), ([100, 130, 64 * c.mb - 7, 9], 2)):
        out = c.run(start=i32(start))
        assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
        for b in range(4):
            assert (out[b * 8:b * 8 + 8] == 0).all() if b == zero else same_bits(out[b * 8:b * 8 + 8], good[b * 8:b * 8 + 8])
    out = c.run(max_ctx=400)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert same_bits(out[:16], good[:16]) and same_bits(out[24:], good[24:])
    for i in range(8):           # depth 2 of sequence 2 is position 512
        row = out[16 + i]
        assert (row == 0).all() if len(tree.path(trees[2], i)) > 2 else same_bits(row, good[16 + i])
    # more nodes than max_nodes, rows outside the call: nothing of the sequence is written
    row0 = i32([0, 8, 24, 24, 32])
    out = c.run(row0=row0)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert (out[8:24] == 7).all() and same_bits(out[:8], good[:8]) and same_bits(out[24:], good[24:])
    out = c.run(row0=i32([0, 8, 16, 24, 33]))
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert (out[24:] == 7).all() and same_bits(out[:24], good[:24])
    # a block id outside the cache
    table = c.table.copy()
    table[1, 0] = c.nb
    out = c.run(table=i32(table))
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert same_bits(out[:8], good[:8]) and torch.isfinite(out).all()


def test_captured_on_another_stream_and_replayed():
    c = Case([make_tree("levels", 12, np.random.default_rng(1))] * 3, [600, 64, 1100], 8, 2, 128, seed=8)
    k, v = c.caches()
    want = c.run(k=k, v=v)
    q = torch.from_numpy(c.q).cuda().to(torch.bfloat16)
    out = torch.zeros_like(want)
    ws = torch.empty(bi.bi_tree_attention_workspace_size(c.T, 8, 128, c.max_ctx, 512), dtype=torch.uint8, device="cuda")
    args = [i32(np.concatenate(c.trees)), i32(c.row0), i32(c.starts), i32(c.table)]

    def call():
        bi.bi_tree_attention(q, c.T, args[0], args[1], args[2], c.B, c.max_nodes, 8, 2, 128, k, v, args[3], c.mb, c.nb,
                             c.max_ctx, 512, c.scale, ws, out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert same_bits(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    other = Case(c.trees, c.starts, 8, 2, 128, seed=31)
    other.table = c.table
    k2, v2 = other.caches()
    for a, b in ((q, torch.from_numpy(other.q).cuda().to(torch.bfloat16)), (k, k2), (v, v2)):
        a.copy_(b)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same_bits(out, other.run())


def test_a_workspace_sixteen_bytes_off():
    c = Case([make_tree("levels", 12, np.random.default_rng(1))] * 2, [600, 1100], 8, 2, 128, seed=8)
    k, v = c.caches()
    q, out = torch.from_numpy(c.q).cuda().to(torch.bfloat16), torch.zeros((c.T, 1024), dtype=torch.bfloat16, device="cuda")
    n = bi.bi_tree_attention_workspace_size(c.T, 8, 128, c.max_ctx, 512)
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")[16:]
    bi.bi_tree_attention(q, c.T, i32(np.concatenate(c.trees)), i32(c.row0), i32(c.starts), c.B, c.max_nodes, 8, 2, 128, k, v,
                         i32(c.table), c.mb, c.nb, c.max_ctx, 512, c.scale, ws, out)
    assert same_bits(out, c.run())


def test_two_calls_at_once_on_two_streams():
    rng = np.random.default_rng(2)
    cs = [Case([make_tree("levels", 20, rng)] * 4, [900, 64, 1500, 7], 8, 2, 128, seed=s) for s in (1, 2)]
    state = [(c.caches(), torch.from_numpy(c.q).cuda().to(torch.bfloat16), c.run()) for c in cs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in cs], [torch.zeros_like(s[2]) for s in state]
    for _ in range(5):
        for c, s, st, o in zip(cs, state, streams, outs):
            with torch.cuda.stream(st):
                c.run(k=s[0][0], v=s[0][1], q=s[1], out=o)
    torch.cuda.synchronize()
    for s, o in zip(state, outs):
        assert same_bits(o, s[2])


def test_a_start_near_the_end_of_the_widest_table():
    c = Case([make_tree("levels", 6, np.random.default_rng(1)), [-1, 0, 0]], [600, 8], 8, 2, 128, seed=8)
    good = c.run()
    k, v = c.caches()
    mb = 0x7fffffff // 64
    table = torch.zeros((2, mb), dtype=torch.int32, device="cuda")
    table[:, :c.mb] = i32(c.table)
    table[1, c.mb:] = int(c.table[1, 0])
    table[1, :c.mb] = int(c.table[1, 0])
    out = torch.full_like(good, 7.0)
    ws = torch.empty(bi.bi_tree_attention_workspace_size(c.T, 8, 128, c.max_ctx, 512), dtype=torch.uint8, device="cuda")
    bi.bi_tree_attention(dev_bf16_from_f32(c.q), c.T, i32(np.concatenate(c.trees)), i32(c.row0), i32([600, mb * 64 - 64]), 2,
                         c.max_nodes, 8, 2, 128, k, v, table, mb, c.nb, c.max_ctx, 512, c.scale, ws, out)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK       # beyond max_ctx: zeros
    assert same_bits(out[:6], good[:6]) and (out[6:] == 0).all()
