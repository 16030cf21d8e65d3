"""Cases of the drafted-rollout operators, in plain form and as calls of the library.

A rollout that drafts sends a tree of candidate tokens per sequence through one step instead of one token.
Five operators serve such a step: the RoPE table of a model (scaled for long contexts or not), the map from
the step's rows to positions (by depth in the tree) and cache slots (by index), the rotation of q and k with
the write of k and v at those slots, attention of every node over the cached context and its own ancestors,
and the acceptance of the longest path that the model agrees with, which moves that path's keys and values
to where the sequence goes on.

`run` computes them with elementary torch operations (`own` false) or with the package's entry points
(`own` true).  A tree is given by `parent` (index of each node's parent within its sequence, -1 for a root,
always below the node's own index), packed over sequences with `row0` as row offsets; node i's key and value
stand in the cache at position start + i, and its own position is start + depth.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 64        # tokens of a cache block
KV_SPLIT = 512    # positions of an attention split
PLAIN, LINEAR, BASE, TURNS, DIMS = range(5)
KINDS = {"plain": PLAIN, "linear": LINEAR, "base": BASE, "turns": TURNS, "dims": DIMS}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the RoPE table of the dense decoder
        dict(name="table_1024x64", op="table", max_pos=1024, rot=64, kind="plain"),
        # a context of 128K tokens reached from 8K by scaling the slow pairs only
        dict(name="table_131072x128_dims", op="table", max_pos=131072, rot=128, kind="dims"),
        # a drafted step of the long-context decoder: 8 nodes a sequence
        dict(name="rope_64x8_hd128", op="rope", B=64, n=8, ctx=2048, Hq=16, Hkv=4, hd=128, rot=128, inter=False, pad=0),
        # larger trees, interleaved pairs on half of each head, qkv rows with a stride of their own
        dict(name="rope_128x64_hd64_part_inter", op="rope", B=128, n=64, ctx=512, Hq=8, Hkv=8, hd=64, rot=32,
             inter=True, pad=8),
        # rows of 16 small trees
        dict(name="slots_16x16", op="slots", B=16, n=16, ctx=768, tree="wide"),
        # rows of 256 chains and trees of up to 64 nodes, empty sequences among them
        dict(name="slots_256x64_ragged", op="slots", B=256, n=64, ctx=8000, tree="ragged"),
        # the dense decoder's rollout batch with 16 nodes a sequence: short contexts, every head its own cache
        dict(name="attn_16x16_ctx768_mha64", op="attn", B=16, n=16, lo=128, hi=768, Hq=8, Hkv=8, hd=64, tree="wide"),
        # one long sequence, 37 nodes: few rows, so the work has to be split over the context
        dict(name="attn_1x37_ctx32768_gqa128", op="attn", B=1, n=37, lo=32768, hi=32768, Hq=16, Hkv=4, hd=128,
             tree="wide"),
        # a serving batch with large trees: 256 query rows share each cached key
        dict(name="attn_16x64_ctx8192_gqa128", op="attn", B=16, n=64, lo=6000, hi=8192, Hq=16, Hkv=4, hd=128,
             tree="wide"),
        # the largest: the long-context decoder's 64 ragged contexts, chains of up to 8 drafted tokens
        dict(name="attn_64x8_ctx32768_gqa128_chain", op="attn", B=64, n=8, lo=1024, hi=32768, Hq=16, Hkv=4, hd=128,
             tree="chain"),
        # the dense decoder's step is accepted: four layers of short rows
        dict(name="accept_16x16_l4_mha64", op="accept", B=16, n=16, ctx=256, layers=4, Hkv=8, hd=64, tree="wide"),
        # 64 sequences of the long-context decoder, trees of 64 nodes
        dict(name="accept_64x64_l8_gqa128", op="accept", B=64, n=64, ctx=400, layers=8, Hkv=4, hd=128, tree="wide"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "slots", "attn", "attn", "attn", "accept", "accept"])
    tree = rng.choice(["wide", "wide", "chain", "ragged"])
    hq, hkv, hd = rng.choice([(8, 8, 64), (16, 4, 128), (16, 4, 128), (4, 2, 64), (16, 2, 128), (12, 12, 128), (16, 1, 64)])
    if op == "table":
        return dict(op=op, max_pos=_log_int(rng, 500, 131072), rot=rng.choice([32, 64, 96, 128]),
                    kind=rng.choice(sorted(KINDS)))
    if op == "rope":
        return dict(op=op, B=_log_int(rng, 1, 128), n=_log_int(rng, 1, 64), ctx=_log_int(rng, 1, 1000), Hq=hq, Hkv=hkv,
                    hd=hd, rot=rng.choice([16, 32, hd // 2, hd, hd]), inter=rng.choice([False, True]),
                    pad=rng.choice([0, 0, 8, 40]))
    if op == "slots":
        return dict(op=op, B=_log_int(rng, 1, 512), n=_log_int(rng, 1, 128), ctx=_log_int(rng, 1, 8000), tree=tree)
    if op == "accept":
        return dict(op=op, B=_log_int(rng, 1, 64), n=_log_int(rng, 1, 64), ctx=_log_int(rng, 1, 400),
                    layers=rng.choice([1, 2, 4, 6]), Hkv=min(hkv, 8), hd=hd, tree=tree)
    while True:
        hi = _log_int(rng, 40, 32768)
        c = dict(op=op, B=_log_int(rng, 1, 64), n=_log_int(rng, 1, 128), lo=rng.choice([0, hi // 8, hi]), hi=hi, Hq=hq,
                 Hkv=hkv, hd=hd, tree=tree)
        if c["B"] * hi * hkv * hd <= 16 * 32768 * 4 * 128 and c["B"] * c["n"] * hq * hi * hd <= 16 * 64 * 16 * 8192 * 128:
            return c


def _trees(case, seed):
    """Host arrays of a drafted step: contexts, nodes per sequence, row offsets and the parent of each node."""
    B, n = case["B"], case["n"]
    # lengths are the case's own; which node is whose child, and every value, go by the seed
    rng = np.random.default_rng([B, n, 11])
    if "hi" in case:   # contexts spread evenly over their logarithm
        ctx = np.exp(rng.uniform(math.log(case["lo"] + 1), math.log(case["hi"] + 1), B)).astype(np.int64) - 1
        ctx = np.clip(ctx, case["lo"], case["hi"])
    else:
        ctx = rng.integers(case["ctx"] // 4, case["ctx"] + 1, B)
    tree = case.get("tree", "wide")
    counts = np.full(B, n)
    if tree in ("ragged", "chain") and n > 1:
        counts = rng.integers(0 if tree == "ragged" else 1, n + 1, B)
        counts[rng.integers(0, B)] = n
    rng = np.random.default_rng([seed, B, n, 13])
    parents = []
    for b in range(B):
        chain = tree == "chain" or (tree == "ragged" and rng.random() < 0.3)
        # a chain, or levels of equal width, each node below one of the level before, as a drafter adds them
        w = 1 if chain else max(2, n // 8)
        parents.append([-1] + [int(rng.integers(max(0, (i - 1) // w * w - w + 1), (i - 1) // w * w + 1))
                               for i in range(1, int(counts[b]))] if counts[b] else [])
    row0 = np.concatenate([[0], np.cumsum(counts)])
    return dict(ctx=ctx, counts=counts, row0=row0, parents=parents, rng=rng)


def _path(parents, i):
    """Nodes from a root down to node i."""
    p = []
    while i >= 0:
        p.append(i)
        i = parents[i]
    return p[::-1]


def work(case):
    op = case["op"]
    if op == "table":
        n = case["max_pos"] * case["rot"]
        return {"bytes": 4 * n, "flops": 2 * n}
    t = _trees(case, 0)
    T, B = int(t["row0"][-1]), case["B"]
    if op == "rope":
        width = (case["Hq"] + 2 * case["Hkv"]) * case["hd"]
        # rows in and out, a position and a slot a row, the table's rows (each position once)
        return {"bytes": T * (4 * width + 12) + min(T, case["ctx"] + case["n"]) * 4 * case["rot"],
                "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if op == "slots":
        return {"bytes": 12 * B + T * (4 + 16) + 4 * int((-(-(t["ctx"] + t["counts"]) // BLOCK) - t["ctx"] // BLOCK).sum()),
                "flops": 4 * T}
    if op == "accept":
        moved, walked = 0, 0
        for b, (path, m) in enumerate(_accepted(case, t)):
            moved += sum(1 for j in range(m) if path[j] != j)
            walked += m
        # tree arrays in, the path out, each moved row's key and value read and written in every layer
        return {"bytes": T * 12 + B * 16 + 8 * walked + moved * case["layers"] * case["Hkv"] * case["hd"] * 2 * 2 * 2,
                "flops": T}
    keys = pairs = 0
    for b in range(B):
        if t["counts"][b]:
            keys += int(t["ctx"][b] + t["counts"][b])
            pairs += int(t["counts"][b]) * int(t["ctx"][b]) + sum(len(_path(t["parents"][b], i)) for i in range(t["counts"][b]))
    # every key and value once, q and the output, the tree
    return {"bytes": keys * case["Hkv"] * case["hd"] * 4 + T * case["Hq"] * case["hd"] * 4 + 4 * T,
            "flops": 4 * pairs * case["Hq"] * case["hd"]}


# ------------------------------------------------------------------------------------ inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _scaling(kind):
    """(factor, trained length, low and high turns, amplitude) of a table's scaling."""
    return {"plain": (1.0, 1.0, 1.0, 2.0, 1.0), "linear": (4.0, 8192.0, 1.0, 2.0, 1.0),
            "base": (4.0, 8192.0, 1.0, 2.0, 1.0), "turns": (8.0, 8192.0, 1.0, 4.0, 1.0),
            "dims": (16.0, 8192.0, 1.0, 32.0, 0.1 * math.log(16.0) + 1.0)}[kind]


def _theta(case):
    return 10000.0 if case["kind"] == "plain" else 500000.0


def _pages(case, t, extra_cols=1):
    """A block table that scatters the sequences' blocks over the cache."""
    need = np.where(t["counts"] > 0, -(-(t["ctx"] + t["counts"]) // BLOCK), -(-t["ctx"] // BLOCK))
    cols = int(need.max()) + extra_cols
    table = np.full((case["B"], cols), -1, np.int32)
    n_blocks = int(need.sum()) + 3
    ids = t["rng"].permutation(n_blocks)[:int(need.sum())]
    table[np.arange(cols)[None, :] < need[:, None]] = ids
    return table, n_blocks


def prepare(case, seed):
    op = case["op"]
    if op == "table":
        s = dict(case=case, table=torch.zeros((case["max_pos"], case["rot"]), device=DEV))
        # the scaling is the model's; a seed moves the base a little, so that other seeds are other tables
        s["theta"] = _theta(case) * (1 + 0.001 * (seed % 97))
        return s
    t = _trees(case, seed)
    T = int(t["row0"][-1])
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + T)
    parent = _i32(np.concatenate([np.asarray(p, np.int32) for p in t["parents"]] or [np.zeros(0, np.int32)]))
    table, n_blocks = _pages(case, t)
    s = dict(case=case, tree=t, T=T, parent=parent, row0=_i32(t["row0"]), start=_i32(t["ctx"]), counts=_i32(t["counts"]),
             table=_i32(table), n_blocks=n_blocks)
    if op == "slots":
        rows = case["B"] * case["n"]     # the buffers' size; rows behind the last sequence stay as they were
        s.update(rows=rows, row0_out=_i32(np.zeros(case["B"] + 1)), row_seq=_i32(np.full(rows, -1)),
                 row_pos=_i32(np.full(rows, -1)), slots=torch.full((rows,), -1, dtype=torch.int64, device=DEV))
        return s

    def bf16(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)

    if op == "rope":
        hq, hkv, hd = case["Hq"], case["Hkv"], case["hd"]
        pos, slots = [], []
        for b, p in enumerate(t["parents"]):
            depth = []
            for i, a in enumerate(p):
                depth.append(0 if a < 0 else depth[a] + 1)
                at = int(t["ctx"][b]) + i
                slots.append(int(table[b, at // BLOCK]) * BLOCK + at % BLOCK)
            pos += [int(t["ctx"][b]) + d for d in depth]
        max_pos = case["ctx"] + case["n"]
        angles = np.arange(max_pos)[:, None] * 10000.0 ** (-2.0 * np.arange(case["rot"] // 2) / case["rot"])
        s.update(qkv=bf16(T, (hq + 2 * hkv) * hd + case["pad"]), pos=_i32(pos), max_pos=max_pos,
                 slots=torch.tensor(slots, dtype=torch.int64, device=DEV),
                 rope=torch.from_numpy(np.concatenate([np.cos(angles), np.sin(angles)], 1).astype(np.float32)).to(DEV),
                 q=torch.zeros((T, hq, hd), dtype=torch.bfloat16, device=DEV),
                 k=torch.zeros((n_blocks, hkv, BLOCK, hd), dtype=torch.bfloat16, device=DEV),
                 v=torch.zeros((n_blocks, hkv, BLOCK, hd), dtype=torch.bfloat16, device=DEV))
        return s
    if op == "accept":
        shape = (case["layers"], n_blocks, case["Hkv"], BLOCK, case["hd"])
        tokens, targets, limit = [], [], []
        for b, (path, m) in enumerate(_accepted(case, t)):
            tok, tgt = t["drafts"][b]
            tokens += tok
            targets += tgt
            limit.append(max(m, 1))
        s.update(tokens=_i32(tokens), targets=_i32(targets), limit=_i32(limit), k=bf16(*shape), v=bf16(*shape),
                 n_out=_i32(np.zeros(case["B"])), pos_out=_i32(np.zeros(case["B"])),
                 path=_i32(np.zeros((case["B"], case["n"]))), out=_i32(np.zeros((case["B"], case["n"]))))
        return s
    hq, hkv, hd = case["Hq"], case["Hkv"], case["hd"]
    # queries that look at some tens of keys among thousands, as trained heads do
    s.update(q=bf16(T, hq, hd, scale=2.0), k=bf16(n_blocks, hkv, BLOCK, hd), v=bf16(n_blocks, hkv, BLOCK, hd),
             scale=1.0 / math.sqrt(hd), max_ctx=int((t["ctx"] + t["counts"]).max()),
             out=torch.zeros((T, hq * hd), dtype=torch.bfloat16, device=DEV))
    if own:
        import invariant_forward_policy_gb300 as bi
        s["ws"] = torch.empty(bi.bi_tree_attention_workspace_size(T, hq, hd, s["max_ctx"], KV_SPLIT),
                              dtype=torch.uint8, device=DEV)
    return s


def _accepted(case, t):
    """(path, length) that each sequence accepts; draws the drafted tokens and the model's choices on the way.

    The model agrees with a drafted child at most nodes.  A length at which moving the path would write over a
    row that a second call of the same step reads again is cut (by `limit`), so that a step can be repeated."""
    rng = np.random.default_rng([int(t["row0"][-1]), sum(sum(p) for p in t["parents"]) + case["B"]])
    t["drafts"], found = [], []
    for p in t["parents"]:
        n = len(p)
        tok = [int(v) for v in rng.integers(0, 32000, n)]
        tgt = [int(v) for v in rng.integers(0, 32000, n)]
        kids = [[] for _ in range(n)]
        for i, a in enumerate(p):
            if a >= 0:
                kids[a].append(i)
        for i in range(n):
            if kids[i] and rng.random() < 0.85:
                at = int(rng.integers(0, len(kids[i])))
                tgt[i] = tok[kids[i][at if i else (0, -1)[at % 2]]]
        t["drafts"].append((tok, tgt))
        path, cur = [], 0 if n else -1
        while cur >= 0:
            path.append(cur)
            cur = next((c for c in kids[cur] if tok[c] == tgt[cur]), -1)
        m = len(path)
        while m and any(path[k] != k and path[k] < m for k in range(m)):
            m -= 1
        found.append((path, m))
    return found


# ------------------------------------------------------------------------------------ plain forms
def _frequencies(case, theta, i):
    """Angle a position of each pair i (64 bits), by the kind of scaling."""
    rot, kind = case["rot"], case["kind"]
    factor, trained, low, high, amp = _scaling(kind)
    if kind == "base":
        theta = theta * factor ** (rot / (rot - 2))
    w = theta ** (-2.0 * i / rot)
    if kind == "linear":
        w = w / factor
    elif kind == "turns":
        keep = torch.clamp((trained * w / (2 * math.pi) - low) / (high - low), 0, 1)
        w = w * keep + w / factor * (1 - keep)
    elif kind == "dims":
        first, last = (rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (high, low))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
        ramp = torch.clamp((i - first) / max(last - first, 0.001), 0, 1)
        w = w * (1 - ramp) + w / factor * ramp
    return w, amp


def _plain_table(s):
    case = s["case"]
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV)
    w, amp = _frequencies(case, s["theta"], i)
    a = torch.arange(case["max_pos"], dtype=torch.float64, device=DEV)[:, None] * w
    return torch.cat([amp * torch.cos(a), amp * torch.sin(a)], 1).float()


def _plain_rope(s):
    c = s["case"]
    T, hq, hkv, hd, rot = s["T"], c["Hq"], c["Hkv"], c["hd"], c["rot"]
    rows = s["qkv"][:, :(hq + 2 * hkv) * hd].view(T, hq + 2 * hkv, hd)
    x = rows[:, :hq + hkv].float()
    cs, sn = s["rope"][s["pos"].long()][:, None].chunk(2, dim=-1)
    y = x.clone()
    if c["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cs - b * sn, b * cs + a * sn
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cs - b * sn, b * cs + a * sn
    y = y.to(torch.bfloat16)
    s["q"].copy_(y[:, :hq])
    s["k"][s["slots"] // BLOCK, :, s["slots"] % BLOCK] = y[:, hq:]
    s["v"][s["slots"] // BLOCK, :, s["slots"] % BLOCK] = rows[:, hq + hkv:]
    return s["q"], s["k"], s["v"]


def _padded(s, a, fill):
    """Packed rows [T] as [B, n] with `fill` behind each sequence's nodes; and where nodes are."""
    i = torch.arange(s["case"]["n"], device=DEV)[None, :]
    there = i < s["counts"][:, None]
    at = torch.clamp(s["row0"][:-1, None].long() + i, max=max(s["T"] - 1, 0))
    return torch.where(there, a[at], fill), there


def _ancestors(parent):
    """[B, n, n]: whether node j is on the path of node i (itself included), by squaring the parent relation."""
    n = parent.shape[1]
    m = (parent[:, :, None] == torch.arange(n, device=DEV)).float() + torch.eye(n, device=DEV)
    steps = 1
    while steps < n:
        m = ((m @ m) > 0).float()
        steps *= 2
    return m > 0


def _plain_slots(s):
    parent, there = _padded(s, s["parent"], -1)
    depth = _ancestors(parent).sum(2) - 1
    n = s["case"]["n"]
    at = s["start"][:, None] + torch.arange(n, device=DEV)
    blk = torch.clamp(at // BLOCK, max=s["table"].shape[1] - 1).long()
    slot = s["table"].gather(1, blk).long() * BLOCK + at % BLOCK
    seq = torch.arange(s["case"]["B"], device=DEV)[:, None].expand(-1, n)
    outs = []
    for a, old in ((seq, s["row_seq"]), (s["start"][:, None] + depth, s["row_pos"]), (slot, s["slots"])):
        new = old.clone()
        new[:s["T"]] = a[there].to(old.dtype)
        outs.append(new)
    row0 = torch.cat([s["counts"].new_zeros(1), s["counts"].cumsum(0).int()])
    return (row0, *outs)


def _plain_attn(s):
    c, t = s["case"], s["tree"]
    hkv, g, hd = c["Hkv"], c["Hq"] // c["Hkv"], c["hd"]
    sees = _ancestors(_padded(s, s["parent"], -1)[0])
    for b in range(c["B"]):
        n, ctx, r0 = int(t["counts"][b]), int(t["ctx"][b]), int(t["row0"][b])
        if not n:
            continue
        pages = s["table"][b, :-(-(ctx + n) // BLOCK)].long()
        k, v = (a[pages].transpose(0, 1).reshape(hkv, -1, hd)[:, :ctx + n].float() for a in (s["k"], s["v"]))
        q = s["q"][r0:r0 + n].float().view(n, hkv, g, hd).permute(1, 0, 2, 3).reshape(hkv, n * g, hd)
        x = (q @ k.transpose(1, 2)) * s["scale"]
        hidden = ~sees[b, :n, :n].repeat_interleave(g, 0)
        x[:, :, ctx:] = x[:, :, ctx:].masked_fill(hidden, -math.inf)
        p = (x - x.max(dim=2, keepdim=True).values).exp()
        o = (p @ v) / p.sum(dim=2, keepdim=True)
        s["out"][r0:r0 + n] = o.view(hkv, n, g, hd).permute(1, 0, 2, 3).reshape(n, -1).to(torch.bfloat16)
    return s["out"]


def _plain_accept(s):
    c = s["case"]
    B, n = c["B"], c["n"]
    parent, there = _padded(s, s["parent"], -1)
    tok, tgt = _padded(s, s["tokens"], -1)[0], _padded(s, s["targets"], -2)[0]
    i = torch.arange(n, device=DEV)
    # first child that carries the token chosen at its parent; n: none
    fits = (parent[:, None, :] == i[None, :, None]) & there[:, None, :] & (tok[:, None, :] == tgt[:, :, None])
    nxt = torch.where(fits, i, n).min(dim=2).values
    cur = torch.where(s["counts"] > 0, 0, n)
    path = torch.full((B, n), -1, dtype=torch.int64, device=DEV)
    for j in range(n):
        ok = (cur < n) & (j < s["limit"])
        path[:, j] = torch.where(ok, cur, -1)
        cur = torch.where(ok, nxt.gather(1, torch.clamp(cur, max=n - 1)[:, None])[:, 0], n)
    on = path >= 0
    m = on.sum(1)
    out = torch.where(on, tgt.gather(1, torch.clamp(path, min=0)), -1)
    b, j = torch.nonzero(on, as_tuple=True)
    src, dst = s["start"][b] + path[b, j], s["start"][b] + j
    blk = [s["table"][b, (a // BLOCK).long()].long() for a in (src, dst)]
    for cache in (s["k"], s["v"]):
        cache[:, blk[1], :, dst % BLOCK] = cache[:, blk[0], :, src % BLOCK]
    return m.int(), path.int(), out.int(), s["start"] + m.int(), s["k"], s["v"]


# ------------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"table": _plain_table, "rope": _plain_rope, "slots": _plain_slots, "attn": _plain_attn,
                "accept": _plain_accept}[op](s)
    import invariant_forward_policy_gb300 as bi
    if op == "table":
        factor, trained, low, high, amp = _scaling(c["kind"])
        bi.bi_rope_scaled_table(s["table"], c["max_pos"], c["rot"], s["theta"],
                                bi.bi_rope_scaling(KINDS[c["kind"]], factor, trained, low, high, amp))
        return s["table"]
    if op == "rope":
        bi.bi_rope_slot_write(s["qkv"], s["T"], s["pos"], s["slots"], c["Hq"], c["Hkv"], c["hd"], s["rope"],
                              s["max_pos"], s["n_blocks"], s["q"], s["k"], s["v"], rot=c["rot"],
                              layout=bi.BI_ROPE_INTERLEAVED if c["inter"] else bi.BI_ROPE_HALF, ld=s["qkv"].shape[1])
        return s["q"], s["k"], s["v"]
    if op == "slots":
        bi.bi_tree_slot_map(s["parent"], s["counts"], s["start"], c["B"], c["n"], s["table"], s["table"].shape[1],
                            s["n_blocks"], s["rows"], s["row0_out"], s["row_seq"], s["row_pos"], s["slots"])
        return s["row0_out"], s["row_seq"], s["row_pos"], s["slots"]
    if op == "attn":
        bi.bi_tree_attention(s["q"], s["T"], s["parent"], s["row0"], s["start"], c["B"], c["n"], c["Hq"], c["Hkv"],
                             c["hd"], s["k"], s["v"], s["table"], s["table"].shape[1], s["n_blocks"], s["max_ctx"],
                             KV_SPLIT, s["scale"], s["ws"], s["out"])
        return s["out"]
    bi.bi_tree_accept(s["parent"], s["row0"], s["start"], s["tokens"], s["targets"], c["B"], c["n"], s["T"], c["n"],
                      s["n_out"], s["path"], s["out"], s["pos_out"], limit=s["limit"], n_layers=c["layers"],
                      Hkv=c["Hkv"], hd=c["hd"], k_cache=s["k"], v_cache=s["v"], block_table=s["table"],
                      max_blocks_per_seq=s["table"].shape[1], n_blocks=s["n_blocks"])
    return s["n_out"], s["path"], s["out"], s["pos_out"], s["k"], s["v"]


# ------------------------------------------------------------------------------------ 64-bit definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "rope": _exact_rope, "slots": _exact_slots, "attn": _exact_attn,
            "accept": _exact_accept}[case["op"]](s)


def _exact_table(s):
    c = s["case"]
    rot, theta = c["rot"], s["theta"]
    factor, trained, low, high, amp = _scaling(c["kind"])
    w = np.empty(rot // 2)
    for i in range(rot // 2):
        f = theta ** (-2.0 * i / rot)
        if c["kind"] == "linear":
            f /= factor
        elif c["kind"] == "base":
            f = (theta * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        elif c["kind"] == "turns":
            part = min(max((trained * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f *= part + (1 - part) / factor
        elif c["kind"] == "dims":
            lo = max(math.floor(rot * math.log(trained / (high * 2 * math.pi)) / (2 * math.log(theta))), 0)
            hi = min(math.ceil(rot * math.log(trained / (low * 2 * math.pi)) / (2 * math.log(theta))), rot - 1)
            part = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f *= (1 - part) + part / factor
        w[i] = f
    turn = np.exp(1j * np.arange(c["max_pos"])[:, None] * w[None, :])
    return np.concatenate([amp * turn.real, amp * turn.imag], axis=1)


def _exact_rope(s):
    c = s["case"]
    hq, hkv, hd, rot = c["Hq"], c["Hkv"], c["hd"], c["rot"]
    x = s["qkv"].double().cpu().numpy()[:, :(hq + 2 * hkv) * hd].reshape(s["T"], hq + 2 * hkv, hd)
    table = s["rope"].double().cpu().numpy()
    pos, slots = s["pos"].cpu().numpy(), s["slots"].cpu().numpy()
    turn = (table[:, :rot // 2] + 1j * table[:, rot // 2:])[pos][:, None, :]
    y = x[:, :hq + hkv].copy()
    pairs = [(2 * j, 2 * j + 1) if c["inter"] else (j, j + rot // 2) for j in range(rot // 2)]
    re, im = [p[0] for p in pairs], [p[1] for p in pairs]
    z = (y[:, :, re] + 1j * y[:, :, im]) * turn
    y[:, :, re], y[:, :, im] = z.real, z.imag
    k, v = (np.zeros((s["n_blocks"], hkv, BLOCK, hd)) for _ in range(2))
    for r in range(s["T"]):
        k[slots[r] // BLOCK, :, slots[r] % BLOCK] = y[r, hq:]
        v[slots[r] // BLOCK, :, slots[r] % BLOCK] = x[r, hq + hkv:]
    return y[:, :hq], k, v


def _exact_slots(s):
    t, table = s["tree"], s["table"].cpu().numpy()
    seq, pos, slot, row0 = [], [], [], [0]
    for b, parents in enumerate(t["parents"]):
        for i in range(len(parents)):
            at = int(t["ctx"][b]) + i
            seq.append(b)
            pos.append(int(t["ctx"][b]) + len(_path(parents, i)) - 1)
            slot.append(int(table[b, at // BLOCK]) * BLOCK + at % BLOCK)
        row0.append(len(seq))
    rest = [-1] * (s["rows"] - len(seq))
    return (np.array(row0, np.int32), np.array(seq + rest, np.int32), np.array(pos + rest, np.int32),
            np.array(slot + rest, np.int64))


def _exact_attn(s):
    c, t = s["case"], s["tree"]
    if s["T"] > 2000:
        return None
    hkv, g, hd = c["Hkv"], c["Hq"] // c["Hkv"], c["hd"]
    out = torch.zeros((s["T"], c["Hq"] * hd), dtype=torch.float64, device=DEV)
    k_all, v_all = (a.transpose(1, 2).reshape(-1, hkv, hd) for a in (s["k"], s["v"]))   # by cache slot
    for b, parents in enumerate(t["parents"]):
        ctx = int(t["ctx"][b])
        place = [int(blk) * BLOCK for blk in s["table"][b].tolist()]
        slot = lambda at: place[at // BLOCK] + at % BLOCK
        old = torch.tensor([slot(a) for a in range(ctx)], dtype=torch.int64, device=DEV)
        k_old, v_old = k_all[old].double(), v_all[old].double()
        for i in range(len(parents)):
            new = torch.tensor([slot(ctx + j) for j in _path(parents, i)], dtype=torch.int64, device=DEV)
            k, v = torch.cat([k_old, k_all[new].double()]), torch.cat([v_old, v_all[new].double()])
            q = s["q"][int(t["row0"][b]) + i].double().view(hkv, g, hd)
            x = torch.einsum("hgd,khd->hgk", q, k) * s["scale"]
            out[int(t["row0"][b]) + i] = torch.einsum("hgk,khd->hgd", torch.softmax(x, -1), v).reshape(-1)
    return out


def _exact_accept(s):
    c, t = s["case"], s["tree"]
    B, n = c["B"], c["n"]
    tok, tgt, table = (s[x].cpu().tolist() for x in ("tokens", "targets", "table"))
    limit = s["limit"].cpu().tolist()
    k, v = s["k"].double().cpu().numpy(), s["v"].double().cpu().numpy()
    count, ends = np.zeros(B, np.int32), np.zeros(B, np.int32)
    paths, outs = np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32)
    for b, parents in enumerate(t["parents"]):
        r0, ctx = int(t["row0"][b]), int(t["ctx"][b])
        path = [0] if parents else []
        while path and len(path) < limit[b]:
            child = [i for i, a in enumerate(parents) if a == path[-1] and tok[r0 + i] == tgt[r0 + path[-1]]]
            if not child:
                break
            path.append(child[0])
        place = lambda at: (table[b][at // BLOCK], at % BLOCK)
        rows = [[a[:, place(ctx + i)[0], :, place(ctx + i)[1]].copy() for i in path] for a in (k, v)]
        for j, i in enumerate(path):
            blk, at = place(ctx + j)
            k[:, blk, :, at], v[:, blk, :, at] = rows[0][j], rows[1][j]
            paths[b, j], outs[b, j] = i, tgt[r0 + i]
        count[b], ends[b] = len(path), ctx + len(path)
    return count, paths, outs, ends, k, v
