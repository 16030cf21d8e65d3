"""Drafted-tree oracle (test infrastructure only): one node at a time, on host lists and in 64 bits.

[Article] §2 (the same discrete choices) and §4.2 (one read path): a step that drafts a tree of tokens gives
each node what plain decoding of its path gives, and keeps the path that plain decoding would have taken.

[Article] is "vLLM Achieves Bitwise-Consistent RL Training: Eliminating Numerical
Drift to Zero KL Divergence on DeepSeek-V4-Flash at 91% Throughput"; section numbers
are its own.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64


def path(parents, i):
    """Nodes from the root down to node i, or None for a node that has no path (a parent that is not before it)."""
    out = []
    while i != -1:
        if not -1 <= parents[i] < i:
            return None
        out.append(i)
        i = parents[i]
    return out[::-1]


def slot_map(trees, start, table):
    """Rows (sequence, position, slot) of the packed trees; position -1 without a path, slot -1 without a block."""
    rows = []
    for b, parents in enumerate(trees):
        for i in range(len(parents)):
            p = path(parents, i)
            at = start[b] + i
            blk = table[b][at // BLOCK] if at // BLOCK < len(table[b]) else -1
            rows.append((b, start[b] + len(p) - 1 if p else -1, blk * BLOCK + at % BLOCK if blk >= 0 else -1))
    return rows


def attention(q, k, v, parents, start, scale):
    """(out, spread) of every node, fp64: q [n, Hq, hd], k and v [start + n, Hkv, hd] by cache position.  spread is the
    mean of |v| under the same weights: what a relative error of the weights is multiplied by."""
    n, hq, hd = q.shape
    g = hq // k.shape[1]
    out, spread = np.zeros((n, hq, hd)), np.zeros((n, hq, hd))
    for i in range(n):
        p = path(parents, i)
        if p is None:
            continue
        at = list(range(start)) + [start + j for j in p]
        for h in range(hq):
            x = k[at, h // g].astype(np.float64) @ q[i, h].astype(np.float64) * scale
            w = np.exp(x - x.max())
            w /= w.sum()
            out[i, h] = w @ v[at, h // g].astype(np.float64)
            spread[i, h] = w @ np.abs(v[at, h // g].astype(np.float64))
    return out, spread


def accept(parents, tokens, targets, limit):
    """Accepted nodes of one sequence: node 0, then the first child that carries the token chosen at the last one."""
    if not len(parents) or parents[0] != -1 or limit < 1:
        return []
    got = [0]
    while len(got) < limit:
        nxt = [i for i, p in enumerate(parents) if p == got[-1] < i and tokens[i] == targets[got[-1]]]
        if not nxt:
            break
        got.append(nxt[0])
    return got


def rope_table(max_pos, rot, theta, kind="plain", factor=1.0, orig_len=1.0, low=1.0, high=2.0, amplitude=1.0):
    """cos then sin of every position and pair, fp64."""
    w = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if kind == "linear":
        w = w / factor
    elif kind == "base":
        w = np.array([(theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)])
    elif kind == "turns":
        keep = np.clip((orig_len * w / (2 * math.pi) - low) / (high - low), 0, 1)
        w = w * (keep + (1 - keep) / factor)
    elif kind == "dims":
        def dim(t):
            return rot * math.log(orig_len / (2 * math.pi * t)) / (2 * math.log(theta))
        a, b = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        r = np.clip((np.arange(rot // 2) - a) / max(b - a, 0.001), 0, 1)
        w = w * (1 - r + r / factor)
    ang = np.arange(max_pos)[:, None] * w
    return np.concatenate([amplitude * np.cos(ang), amplitude * np.sin(ang)], axis=1)


def rotate(x, cos, sin, rot, interleaved):
    """Heads x [.., hd] turned by one angle a pair, every product and sum rounded to fp32 (then to bf16 by the caller)."""
    x, cos, sin = x.astype(np.float32), cos.astype(np.float32), sin.astype(np.float32)
    y = x.copy()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y
