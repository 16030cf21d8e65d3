"""Paged-cache planning oracle (test infrastructure only): one request at a time on host lists.

[Article] §4.2: every phase reads and writes K/V through a block table; a position p of a request
lives in block table[p // 64], slot p % 64.  The pool of free blocks is a queue.

[Article] is "vLLM Achieves Bitwise-Consistent RL Training: Eliminating Numerical
Drift to Zero KL Divergence on DeepSeek-V4-Flash at 91% Throughput"; section numbers
are its own.
"""
from __future__ import annotations

from collections import deque

BLOCK = 64


def resize(lens, extra, table, owned, free):
    """New (table, owned, free queue, failed requests): `table` is a list of lists of exactly max_blocks
    entries (-1 unused), `free` the free ids in the order in which they are handed out.  Ids that a call
    gives back are not handed out by it."""
    table, owned, free = [list(r) for r in table], list(owned), deque(free)
    room, asked, failed, back = len(free), 0, [], []
    for b, n in enumerate(lens):
        need = -(-(n + extra) // BLOCK) if n > 0 else 0
        if need > len(table[b]):
            failed.append(b)
            continue
        if need < owned[b]:
            for i in range(need, owned[b]):
                back.append(table[b][i])
                table[b][i] = -1
            owned[b] = need
            continue
        more = need - owned[b]
        asked += more
        if more and asked > room:
            failed.append(b)
            continue
        for i in range(owned[b], need):
            table[b][i] = free.popleft()
        owned[b] = need
    return table, owned, list(free) + back, failed


def slot_map(new, start, table, T):
    """(row0, rows): rows are (request, position, slot) of the first T packed rows, slot -1 without a block."""
    row0, rows = [0], []
    for b, n in enumerate(new):
        for p in range(start[b], start[b] + n):
            blk = table[b][p // BLOCK] if 0 <= p < BLOCK * len(table[b]) else -1
            rows.append((b, p, blk * BLOCK + p % BLOCK if blk >= 0 else -1))
        row0.append(min(T, len(rows)))
    return row0, rows[:T]
