"""Refusals of the drafted-tree and RoPE entry points: every bad argument is answered on the host before
anything is launched (dummy addresses; no GPU is reached)."""
import ctypes
import math

import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300 import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="passes dummy addresses: a regressed check must not be able to launch")
INVALID, SHAPE = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_rope_scaled_table(lib):
    def call(table=16, max_pos=100, rot=64, theta=1e4, **s):
        return lib.bi_rope_scaled_table(table, max_pos, rot, theta, ctypes.byref(bi.bi_rope_scaling(**s)) if s else None,
                                        None)
    assert call(table=None) == INVALID and "null" in bi.bi_last_error()
    for bad in (dict(max_pos=0), dict(max_pos=(1 << 31) + 1), dict(rot=63), dict(rot=0), dict(rot=-2), dict(theta=1.0),
                dict(theta=math.nan), dict(theta=math.inf), dict(kind=5), dict(kind=-1), dict(amplitude=math.nan),
                dict(amplitude=1e300), dict(kind=bi.BI_ROPE_LINEAR, factor=0.0), dict(kind=bi.BI_ROPE_LINEAR, factor=math.nan),
                dict(kind=bi.BI_ROPE_BASE, rot=2, factor=2.0), dict(kind=bi.BI_ROPE_BASE, rot=4, factor=1e-9),
                dict(kind=bi.BI_ROPE_TURNS, factor=2.0, low=4.0, high=4.0),
                dict(kind=bi.BI_ROPE_TURNS, factor=2.0, low=0.0, high=4.0),
                dict(kind=bi.BI_ROPE_DIMS, factor=2.0, orig_len=0.0), dict(kind=bi.BI_ROPE_DIMS, factor=2.0, high=math.inf)):
        assert call(**bad) == INVALID, bad
    assert call(rot=258) == SHAPE
    for kind in (bi.BI_ROPE_LINEAR, bi.BI_ROPE_TURNS, bi.BI_ROPE_DIMS):      # angles beyond the range of doubles
        assert call(kind=kind, factor=5e-324) == INVALID and "finite" in bi.bi_last_error()


def test_rope_slot_write(lib):
    def call(qkv=16, T=4, ld=1024, pos=16, slots=16, Hq=8, Hkv=4, hd=64, rot=64, layout=0, table=16, max_pos=10, nb=3,
             q=16, k=16, v=16):
        return lib.bi_rope_slot_write(qkv, T, ld, pos, slots, Hq, Hkv, hd, rot, layout, table, max_pos, nb, q, k, v, None)
    assert call(T=0, qkv=None, q=None) == bi.BI_OK
    for name in ("qkv", "pos", "slots", "table", "q", "k", "v"):
        assert call(**{name: None}) == INVALID, name
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=-1), dict(hd=0), dict(max_pos=0), dict(nb=0), dict(layout=2), dict(rot=80),
                dict(rot=-16), dict(ld=1023), dict(qkv=24), dict(k=20), dict(table=8), dict(T=1 << 31)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(hd=60, rot=16), dict(rot=24), dict(rot=20, layout=1), dict(ld=1028), dict(hd=2048, ld=1 << 20)):
        assert call(**bad) == SHAPE, bad
    assert "multiple" in bi.bi_last_error() or "at most" in bi.bi_last_error()


def test_tree_slot_map(lib):
    def call(parent=16, counts=16, start=16, B=2, most=8, table=16, mb=4, nb=9, T=16, row0=16, seq=None, pos=None, slots=16):
        return lib.bi_tree_slot_map(parent, counts, start, B, most, table, mb, nb, T, row0, seq, pos, slots, None)
    assert call(B=0, counts=None, row0=None) == bi.BI_OK
    for bad in (dict(B=-1), dict(T=-1), dict(parent=None), dict(counts=None), dict(start=None), dict(row0=None),
                dict(table=None), dict(most=0), dict(mb=0), dict(nb=0), dict(B=1 << 21), dict(T=1 << 31)):
        assert call(**bad) == INVALID, bad
    assert call(most=257) == SHAPE


def test_tree_attention(lib):
    def call(q=16, T=8, parent=16, row0=16, start=16, B=2, most=8, Hq=8, Hkv=4, hd=64, k=16, v=16, table=16, mb=4, nb=9,
             ctx=256, split=512, ws=16, size=1 << 30, out=16):
        return lib.bi_tree_attention(q, T, parent, row0, start, B, most, Hq, Hkv, hd, k, v, table, mb, nb, ctx, split, 0.1,
                                     ws, size, out, None)
    assert call(T=0, q=None) == bi.BI_OK and call(B=0, out=None) == bi.BI_OK
    for name in ("q", "parent", "row0", "start", "k", "v", "table", "ws", "out"):
        assert call(**{name: None}) == INVALID, name
    for bad in (dict(T=-1), dict(B=-1), dict(most=0), dict(Hq=0), dict(Hkv=3), dict(split=100), dict(split=0), dict(ctx=0),
                dict(mb=0), dict(nb=0), dict(q=18), dict(ws=8), dict(k=4), dict(B=65536), dict(ctx=64 * 70000, split=64)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(most=257), dict(hd=96), dict(Hq=12, Hkv=4), dict(Hq=256, Hkv=2), dict(split=16448),
                dict(nb=1 << 24), dict(mb=1 << 26)):
        assert call(**bad) == SHAPE, bad
    need = 8 * 8 * 1 * 66 * 4 + 8 * 4
    assert bi.bi_tree_attention_workspace_size(8, 8, 64, 256, 512) >= need
    assert call(size=need - 1) == INVALID and "workspace" in bi.bi_last_error()
    assert bi.bi_tree_attention_workspace_size(0, 8, 64, 256, 512) == 0


def test_tree_accept(lib):
    def call(parent=16, row0=16, start=1 << 20, tokens=16, targets=16, limit=None, B=2, most=8, T=8, path_len=8, n=16,
             path=16, out=16, pos=1 << 21, layers=2, Hkv=4, hd=64, k=16, v=16, table=16, mb=4, nb=9):
        return lib.bi_tree_accept(parent, row0, start, tokens, targets, limit, B, most, T, path_len, n, path, out, pos,
                                  layers, Hkv, hd, k, v, table, mb, nb, None)
    assert call(B=0, row0=None, n=None) == bi.BI_OK
    for name in ("parent", "row0", "start", "tokens", "targets", "n", "path", "out", "pos", "k", "v", "table"):
        assert call(**{name: None}) == INVALID, name
    for bad in (dict(B=-1), dict(T=-1), dict(most=0), dict(path_len=0), dict(B=65536), dict(path_len=1 << 31),
                dict(pos=1 << 20), dict(pos=(1 << 20) + 4), dict(layers=0), dict(Hkv=0), dict(hd=0), dict(mb=0), dict(nb=0),
                dict(k=8)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(most=257), dict(hd=60), dict(nb=1 << 31), dict(layers=5000)):
        assert call(**bad) == SHAPE, bad
