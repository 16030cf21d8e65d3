"""Inputs of the drafted-tree GPU tests: trees, paged caches whose other slots hold NaN, and the linear form
of every node's path for bi_attention."""
import numpy as np
import torch

import invariant_forward_policy_gb300 as bi
from gpu_util import dev_bf16_from_f32
from oracle import tree


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def make_tree(kind, n, rng):
    """Parents of n nodes: a chain, levels of equal width, random attachment, or a forest of several roots."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "levels":
        w = max(2, n // 6)
        return [-1] + [int(rng.integers(max(0, (i - 1) // w * w - w + 1), (i - 1) // w * w + 1)) for i in range(1, n)]
    low = -1 if kind == "forest" else 0
    return ([-1] + [int(rng.integers(low, i)) for i in range(1, n)])[:n]


class Case:
    """Trees over a paged cache: `starts` tokens before each, all other cache slots NaN."""

    def __init__(self, trees, starts, hq, hkv, hd, seed=0, extra_rows=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.trees, self.starts, self.hq, self.hkv, self.hd = trees, starts, hq, hkv, hd
        self.B, self.max_nodes = len(trees), max(1, max(len(t) for t in trees))
        self.row0 = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32)
        self.T = int(self.row0[-1])
        need = [-(-(s + len(t)) // 64) for s, t in zip(starts, trees)]
        self.mb = max(1, max(need))
        self.nb = sum(need) + 2
        ids = rng.permutation(self.nb)
        self.table = np.full((self.B, self.mb), -1, np.int32)
        o = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[o:o + m]
            o += m
        bf = lambda x: torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()
        self.k = [bf(rng.normal(size=(s + len(t), hkv, hd))) for s, t in zip(starts, trees)]   # by cache position
        self.v = [bf(rng.normal(size=(s + len(t), hkv, hd))) for s, t in zip(starts, trees)]
        self.q = bf(rng.normal(size=(self.T + extra_rows, hq, hd)) * qscale)
        self.scale = 1.0 / np.sqrt(hd)
        self.max_ctx = max(1, max(s + len(t) for s, t in zip(starts, trees)))

    def caches(self):
        out = []
        for src in (self.k, self.v):
            c = np.full((self.nb, self.hkv, 64, self.hd), np.nan, np.float32)
            for b, x in enumerate(src):
                for p in range(len(x)):
                    c[self.table[b, p // 64], :, p % 64] = x[p]
            out.append(dev_bf16_from_f32(c))
        return out

    def run(self, split=512, k=None, v=None, out=None, q=None, parent=None, start=None, row0=None, table=None, T=None,
            max_ctx=None, max_nodes=None):
        if k is None:
            k, v = self.caches()
        T = self.T if T is None else T
        max_ctx = self.max_ctx if max_ctx is None else max_ctx
        q = dev_bf16_from_f32(self.q) if q is None else q
        if parent is None:
            parent = i32(np.concatenate([np.asarray(t, np.int32) for t in self.trees]))
        if out is None:
            out = torch.full((T, self.hq * self.hd), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((bi.bi_tree_attention_workspace_size(T, self.hq, self.hd, max_ctx, split) // 4 + 1,), float("nan"),
                        device="cuda").view(torch.uint8)
        bi.bi_tree_attention(q, T, parent, i32(self.row0) if row0 is None else row0,
                             i32(self.starts) if start is None else start, self.B,
                             self.max_nodes if max_nodes is None else max_nodes, self.hq, self.hkv, self.hd, k, v,
                             i32(self.table) if table is None else table, self.mb, self.nb, max_ctx, split, self.scale, ws,
                             out)
        return out

    def linear(self, split=512):
        """bi_attention of every node on a cache of its own that holds just its path (a decode step each)."""
        pages, tab, pos = [], [], []
        mb = -(-self.max_ctx // 64)
        for b, t in enumerate(self.trees):
            for i in range(len(t)):
                at = list(range(self.starts[b])) + [self.starts[b] + j for j in tree.path(t, i)]
                n = -(-len(at) // 64)
                row = np.full(mb, -1, np.int32)
                for p in range(n):
                    row[p] = len(pages)
                    sel = at[p * 64:(p + 1) * 64]
                    page = np.full((2, self.hkv, 64, self.hd), np.nan, np.float32)
                    page[0, :, :len(sel)] = self.k[b][sel].transpose(1, 0, 2)
                    page[1, :, :len(sel)] = self.v[b][sel].transpose(1, 0, 2)
                    pages.append(page)
                tab.append(row)
                pos.append(len(at) - 1)
        T = self.T
        pages = np.stack(pages)
        k, v = dev_bf16_from_f32(pages[:, 0]), dev_bf16_from_f32(pages[:, 1])
        out = torch.empty((T, self.hq * self.hd), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(bi.bi_attention_workspace_size(T, self.hq, self.hd, self.max_ctx, split), dtype=torch.uint8,
                         device="cuda")
        bi.bi_attention(dev_bf16_from_f32(self.q[:T]), T, i32(np.arange(T)), i32(np.arange(T + 1)), i32(pos), T, 1, self.hq,
                        self.hkv, self.hd, k, v, i32(np.stack(tab)), mb, len(pages), self.max_ctx, split, self.scale, ws,
                        out)
        return out
