"""Pins of the drafted-tree oracle: hand-worked trees, the causal form, and the RoPE table's closed forms."""
import math

import numpy as np

from oracle import ops, tree


def test_paths_positions_and_slots_by_hand():
    #        0
    #      1   2
    #     3     4 5     6 is a second root, 7 stands under it
    parents = [-1, 0, 0, 1, 2, 2, -1, 6]
    assert [tree.path(parents, i) for i in (0, 3, 5, 7)] == [[0], [0, 1, 3], [0, 2, 5], [6, 7]]
    assert tree.path([0], 0) is None and tree.path([-1, 2, 0], 1) is None and tree.path([-1, 1, 1], 2) is None
    rows = tree.slot_map([parents, [-1]], [62, 0], [[9, 4], [-1, -1]])
    assert [r[1] for r in rows] == [62, 63, 63, 64, 64, 64, 62, 63, 0]
    assert [r[2] for r in rows[:3]] == [9 * 64 + 62, 9 * 64 + 63, 4 * 64] and rows[-1][2] == -1


def test_a_chain_is_causal_attention_and_siblings_do_not_meet():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(4, 2, 8)), rng.normal(size=(9, 1, 8)), rng.normal(size=(9, 1, 8))
    want = ops.attention(q.astype(np.float32), k.astype(np.float32), v.astype(np.float32), np.arange(5, 9))
    got, spread = tree.attention(q, k, v, [-1, 0, 1, 2], 5, 1 / math.sqrt(8))
    # ops.attention rounds its output to bf16: at most 2^-8 of the value
    np.testing.assert_allclose(got, np.asarray(want).reshape(got.shape), rtol=2.0**-8, atol=1e-5)
    assert (spread >= np.abs(got) - 1e-12).all()
    # node 2 is a child of node 0: node 1's key and value do not matter to it
    a = tree.attention(q, k, v, [-1, 0, 0, 2], 5, 0.3)[0]
    k2, v2 = k.copy(), v.copy()
    k2[6], v2[6] = np.nan, np.nan
    b = tree.attention(q, k2, v2, [-1, 0, 0, 2], 5, 0.3)[0]
    assert (a[[0, 2, 3]] == b[[0, 2, 3]]).all() and np.isnan(b[1]).all()


def test_acceptance_by_hand():
    parents, tokens = [-1, 0, 0, 2, 2, 4], [7, 1, 2, 3, 3, 9]
    assert tree.accept(parents, tokens, [2, 0, 3, 9, 9, 5], 10) == [0, 2, 3]       # the first of two equal children
    assert tree.accept(parents, tokens, [2, 0, 3, 0, 9, 5], 2) == [0, 2]
    assert tree.accept(parents, tokens, [4, 0, 3, 0, 9, 5], 9) == [0]
    assert tree.accept([], [], [], 3) == [] and tree.accept([-1], [1], [1], 0) == [] and tree.accept([0], [1], [1], 2) == []


def test_rope_table_forms():
    plain = tree.rope_table(64, 16, 10000.0)
    np.testing.assert_allclose(plain[:, :8] ** 2 + plain[:, 8:] ** 2, 1, atol=1e-14)
    cos, sin = ops.rope_cos_sin(np.arange(64), 16)
    np.testing.assert_allclose(plain, np.concatenate([cos, sin], 1), atol=1e-6)
    # positions interpolated: entry 4 p is the plain entry p
    np.testing.assert_allclose(tree.rope_table(64, 16, 1e4, "linear", 4.0)[::4], plain[:16], atol=1e-12)
    # the slowest pair of a scaled base turns factor times slower, the fastest as before
    base = tree.rope_table(4, 16, 1e4, "base", 4.0)
    w = np.arctan2(base[1, 8:], base[1, :8])
    assert abs(w[0] - 1) < 1e-12 and abs(w[7] * 4 - 1e4 ** (-14 / 16)) < 1e-12
    for kind in ("turns", "dims"):
        t = tree.rope_table(2, 64, 1e4, kind, 8.0, 4096.0, 1.0, 32.0)
        w = np.arctan2(t[1, 32:], t[1, :32]) / (1e4 ** (-np.arange(32) / 32))
        assert abs(w[0] - 1) < 1e-9 and abs(w[-1] - 1 / 8) < 1e-9 and (np.diff(w) < 1e-9).all()
    x = np.random.default_rng(1).normal(size=(3, 16)).astype(np.float32)
    full = tree.rotate(x, plain[5, :8], plain[5, 8:], 16, False)
    inter = tree.rotate(x.reshape(3, 2, 8).transpose(0, 2, 1).reshape(3, 16), plain[5, :8], plain[5, 8:], 16, True)
    assert (inter.reshape(3, 8, 2).transpose(0, 2, 1).reshape(3, 16) == full).all()
    part = tree.rotate(x, plain[5, :4], plain[5, 8:12], 8, False)
    assert (part[:, 8:] == x[:, 8:]).all()
