"""bi_tree_attention refuses a workspace that lacks a byte of its split or tail records, or of what an address that is
16-byte but not 32-byte aligned skips (dummy addresses; no GPU is reached)."""
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from invariant_forward_policy_gb300 import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="passes dummy addresses: a regressed check must not be able to launch")


def _lanes_behind(nodes, split):
    """The most lanes (a quarter of a split in whole 64s; a split's last one may be shorter) that `nodes` positions meet."""
    lane = -(-split // 256) * 64
    edges = sorted({s * split + j for s in range(2 + -(-2 * nodes // split)) for j in range(0, split, lane)})
    return max(sum(p < e <= p + nodes - 1 for e in edges) + 1 for p in range(split))


def _bytes(T, Hq, hd, ctx, split, nodes):
    return T * Hq * (-(-ctx // split) + _lanes_behind(nodes, split)) * (hd + 2) * 4 + T * 4


# at `nodes` the count of tail records that a call sets aside is the least there can be
@pytest.mark.parametrize("T,Hq,Hkv,hd,ctx,split,nodes", [(8, 8, 4, 64, 256, 512, 8), (5, 2, 1, 128, 6000, 512, 2),
                                                         (300, 16, 4, 128, 9000, 64, 129), (7, 4, 4, 64, 1, 1024, 1)])
@pytest.mark.parametrize("ws,skip", [(32, 0), (16, 16), (48, 16), (1 << 20, 0)])
def test_one_byte_short(T, Hq, Hkv, hd, ctx, split, nodes, ws, skip):
    need = _bytes(T, Hq, hd, ctx, split, nodes) + skip
    status = _lib.load().bi_tree_attention(16, T, 16, 16, 16, 1, nodes, Hq, Hkv, hd, 16, 16, 16, 200, 9, ctx, split, 0.1, ws,
                                           need - 1, 16, None)
    assert status == bi.BI_ERR_INVALID_ARG and "workspace" in bi.bi_last_error()


@pytest.mark.parametrize("split", [64, 128, 320, 512, 576, 832, 1024, 16384])
@pytest.mark.parametrize("T,Hq,hd,ctx", [(1, 1, 64, 1), (8, 8, 64, 256), (4096, 16, 128, 32768)])
def test_the_size_holds_every_call(T, Hq, hd, ctx, split):
    assert bi.bi_tree_attention_workspace_size(T, Hq, hd, ctx, split) >= _bytes(T, Hq, hd, ctx, split, 256) + 16
