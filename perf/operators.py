"""Cases of the sampling and paged-cache planning operators, in plain form and as calls of the library.

Four operators of one decode step that samples: the draw of a token from a row of logits
(temperature, min-p, top-k, top-p, given random numbers), the logprob of given tokens under the
same truncated distribution (the training recompute's side of it), the block tables of a paged KV
cache resized to the requests' lengths, and the map from a step's rows to sequences, positions and
cache slots.

`run` computes them with elementary torch operations (`own` false) or with the package's entry
points (`own` true).  Token choices sit next to borders of a cumulative sum, so the plain form
works in 64 bits and rounds the logprob once at the end.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 64                    # tokens of a cache block
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
MOST_LOGITS = 2048 * 129280   # elements of the largest listed case


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence's decode step on a small vocabulary: latency alone
        dict(name="sample_1x4096_topk", op="sample", T=1, V=4096, pad=0, dtype="fp32", shape="peaked", rule="topk"),
        # the dense decoder's rollout batch, sampled at its temperature with nothing cut off
        dict(name="sample_16x32000_temp", op="sample", T=16, V=32000, pad=0, dtype="fp32", shape="flat", rule="temp"),
        # a serving batch over a large vocabulary, top-k then top-p
        dict(name="sample_64x129280_topk_topp", op="sample", T=64, V=129280, pad=0, dtype="fp32", shape="peaked",
             rule="topk_topp"),
        # nucleus sampling with no top-k: the mass of the whole row decides where it is cut
        dict(name="sample_256x129280_topp", op="sample", T=256, V=129280, pad=0, dtype="fp32", shape="peaked",
             rule="topp"),
        # an odd vocabulary in bf16 with padded rows, every request with a rule of its own (greedy ones among them)
        dict(name="sample_37x50261_mixed_bf16", op="sample", T=37, V=50261, pad=3, dtype="bf16", shape="peaked",
             rule="mixed"),
        # the training recompute of the dense decoder's 16 x 256 generated tokens under top-p
        dict(name="logprob_4096x32000_topp", op="logprob", T=4096, V=32000, pad=0, dtype="fp32", shape="flat",
             rule="topp"),
        # scoring over a large vocabulary, temperature only
        dict(name="logprob_512x129280_temp", op="logprob", T=512, V=129280, pad=0, dtype="fp32", shape="peaked",
             rule="temp"),
        # the largest: a packed recompute's rows in bf16, min-p, top-k and top-p mixed
        dict(name="logprob_2048x129280_mixed_bf16", op="logprob", T=2048, V=129280, pad=0, dtype="bf16",
             shape="peaked", rule="mixed"),
        # a decode step of 64 long-context sequences: about one in 64 crosses into a new block
        dict(name="blocks_64_decode", op="blocks", B=64, max_blocks=512, mean_ctx=9000, new="one"),
        # a scheduler admitting and growing thousands of requests in chunks
        dict(name="blocks_4096_admit", op="blocks", B=4096, max_blocks=512, mean_ctx=8000, new="chunk"),
        # the same decode step's rows: one token each
        dict(name="slots_64_decode", op="slots", B=64, max_blocks=512, mean_ctx=9000, new="one"),
        # a packed chunked-prefill step: ragged pieces of up to 2048 tokens, decode rows and empty requests among them
        dict(name="slots_256_prefill", op="slots", B=256, max_blocks=512, mean_ctx=8000, new="chunk"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "logprob", "logprob", "blocks", "slots"])
    if op in ("sample", "logprob"):
        V = _log_int(rng, 1000, 160000)
        T = _log_int(rng, 1, min(1024 if op == "sample" else 8192, MOST_LOGITS // V))
        return dict(op=op, T=T, V=V, pad=rng.choice([0, 0, 1, 5, 8]), dtype=rng.choice(["fp32", "fp32", "bf16"]),
                    shape=rng.choice(["flat", "peaked", "peaked"]),
                    rule=rng.choice(["temp", "topk", "topp", "minp", "topk_topp", "mixed"]))
    return dict(op=op, B=_log_int(rng, 1, 4096 if op == "blocks" else 512), max_blocks=_log_int(rng, 16, 512),
                mean_ctx=_log_int(rng, 64, 8000), new=rng.choice(["one", "chunk"]))


def work(case):
    """Bytes: every input and output once.  Operations: per logit a difference, a scaling, an exponential and a sum."""
    if case["op"] in ("sample", "logprob"):
        n = case["T"] * case["V"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["T"] * 28, "flops": 4 * n}
    plan = _lengths(case, 0)
    if case["op"] == "blocks":
        grown = int((plan["need"] - plan["owned"]).sum())
        # lengths, owned counts in and out; each new block's id read from the pool and written to the table
        return {"bytes": 12 * case["B"] + 8 * grown + 16, "flops": 4 * case["B"] + 2 * grown}
    rows = int(plan["new"].sum())
    # lengths and starts in, row offsets out; per row its sequence, position and slot, and each block id that is read
    blocks = int((-(-(plan["ctx"] + plan["new"]) // BLOCK) - plan["ctx"] // BLOCK)[plan["new"] > 0].sum())
    return {"bytes": 12 * case["B"] + 16 * rows + 4 * blocks, "flops": 4 * case["B"] + 4 * rows}


# ------------------------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """Host arrays of a step: tokens in the cache (ctx), tokens that the step adds (new), blocks owned and needed."""
    rng = np.random.default_rng([seed, case["B"], case["max_blocks"]])
    B, most = case["B"], case["max_blocks"] * BLOCK
    ctx = np.clip(rng.lognormal(math.log(case["mean_ctx"]), 0.6, B), 1, most - 1).astype(np.int64)
    if case["new"] == "one":
        new = np.ones(B, np.int64)
    else:
        kind = rng.random(B)
        new = rng.integers(1, 2049, B)
        new[kind < 0.2] = 1
        new[(kind >= 0.2) & (kind < 0.3)] = 0
        ctx[kind > 0.7] = 0          # newly admitted requests
    new = np.minimum(new, most - ctx)
    # the step's token budget is fixed: the last requests get what is left of it
    budget = B if case["new"] == "one" else 900 * B
    new = np.clip(budget - (np.cumsum(new) - new), 0, new)
    owned = -(-ctx // BLOCK)
    need = np.maximum(owned, -(-(ctx + new) // BLOCK))
    return dict(ctx=ctx, new=new, owned=owned, need=need, rng=rng, budget=budget)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _params(case, seed):
    """Per-row sampling parameters of the case's rule (host)."""
    rng = np.random.default_rng([seed, 7])
    T = case["T"]
    temp = rng.uniform(0.6, 1.2, T).astype(np.float32)
    k = rng.choice([5, 20, 40, 50, 64, 200], T).astype(np.int32)
    p = rng.choice([0.8, 0.9, 0.95, 0.99], T).astype(np.float32)
    mp = rng.choice([0.01, 0.05, 0.1], T).astype(np.float32)
    rule = case["rule"]
    use_k = np.isin(rule, ["topk", "topk_topp"]) | np.zeros(T, bool)
    use_p = np.isin(rule, ["topp", "topk_topp"]) | np.zeros(T, bool)
    use_m = (rule == "minp") | np.zeros(T, bool)
    if rule == "mixed":
        use_k, use_p, use_m = rng.random(T) < 0.4, rng.random(T) < 0.5, rng.random(T) < 0.3
        temp[rng.random(T) < 0.1] = 0.0
    return (temp, np.where(use_k, k, 0).astype(np.int32), np.where(use_p, p, 1).astype(np.float32),
            np.where(use_m, mp, 0).astype(np.float32))


def prepare(case, seed):
    if case["op"] in ("blocks", "slots"):
        return _prepare_pages(case, seed)
    T, V, ld = case["T"], case["V"], case["V"] + case["pad"]
    g = torch.Generator(device=DEV).manual_seed(seed * 1009 + T)
    # peaked: a model's logits, a broad body with some tens of likely tokens; flat: those of random weights
    x = torch.randn((T, ld), generator=g, device=DEV) * (2.5 if case["shape"] == "peaked" else 1.0)
    if case["shape"] == "peaked":
        at = torch.randint(0, V, (T, 32), generator=g, device=DEV)
        x.scatter_(1, at, 3.0 + 15.0 * torch.rand((T, 32), generator=g, device=DEV))
    logits = x.to(DTYPES[case["dtype"]])
    temp, k, p, mp = (torch.from_numpy(a).to(DEV) for a in _params(case, seed))
    s = dict(case=case, logits=logits, temp=temp, k=k, p=p, mp=mp,
             u=torch.rand(T, generator=g, device=DEV),
             out_ids=torch.zeros(T, dtype=torch.int32, device=DEV),
             out_lp=torch.zeros(T, dtype=torch.float32, device=DEV))
    if case["op"] == "logprob":   # the tokens that a rollout drew from these rows
        s["ids"] = _plain_sample(s)[0]
    return s


def _prepare_pages(case, seed):
    pl = _lengths(case, seed)
    rng, B, mb = pl["rng"], case["B"], case["max_blocks"]
    n_owned, n_need = int(pl["owned"].sum()), int(pl["need"].sum())
    n_blocks = n_need + n_need // 8 + 16
    ids = rng.permutation(n_blocks).astype(np.int32)
    have = np.arange(mb)[None, :] < pl["owned"][:, None]
    table = np.full((B, mb), -1, np.int32)
    s = dict(case=case, n_blocks=n_blocks)
    if case["op"] == "blocks":
        table[have] = ids[:n_owned]
        # the free blocks stand in a ring from a place of their own
        ring = np.full(n_blocks, -1, np.int32)
        head = int(rng.integers(0, n_blocks))
        ring[(head + np.arange(n_blocks - n_owned)) % n_blocks] = ids[n_owned:]
        s.update(lens=_i32(pl["ctx"] + pl["new"]), table=_i32(table), owned=_i32(pl["owned"]), ring=_i32(ring),
                 pool=_i32([head, n_blocks - n_owned]), owned_out=_i32(np.zeros(B)), pool_out=_i32([0, 0]))
        return s
    table[np.arange(mb)[None, :] < pl["need"][:, None]] = ids[:n_need]
    rows = pl["budget"]   # the buffers' size; rows behind the last sequence stay as they were
    s.update(new=_i32(pl["new"]), start=_i32(pl["ctx"]), table=_i32(table), rows=rows, row0=_i32(np.zeros(B + 1)),
             row_seq=_i32(np.full(rows, -1)), row_pos=_i32(np.full(rows, -1)),
             slots=torch.full((rows,), -1, dtype=torch.int64, device=DEV))
    return s


# ------------------------------------------------------------------------------------ plain forms
def _plain_rows(s):
    """(scaled logits, kept mask, mass of the kept tokens with 0 elsewhere), in 64 bits and in index order."""
    V = s["case"]["V"]
    x = s["logits"][:, :V].double()
    greedy = s["temp"] == 0
    T = torch.where(greedy, 1.0, s["temp"]).double()[:, None]
    k = torch.where(greedy, 1, torch.where((s["k"] <= 0) | (s["k"] > V), V, s["k"]))[:, None]
    p = torch.where(greedy, 1.0, s["p"]).double()[:, None]
    z = (x - x.max(dim=1, keepdim=True).values) / T
    w = z.exp()
    # larger logits first, ties to the lower index
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    allowed = (ws > 0) & (ws >= s["mp"].double()[:, None]) & (torch.arange(V, device=x.device)[None, :] < k)
    ws = torch.where(allowed, ws, 0.0)
    through = ws.cumsum(dim=1)
    before = through - ws
    keep = allowed & ((p >= 1) | (before < p * through[:, -1:]))
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    return z, kept, torch.where(kept, w, 0.0)


def _plain_sample(s):
    z, kept, w = _plain_rows(s)
    cum = w.cumsum(dim=1)
    total = cum[:, -1:]
    ids = (cum <= s["u"].double()[:, None] * total).sum(dim=1, keepdim=True)
    lp = z.gather(1, ids) - total.log()
    return ids[:, 0].int(), lp[:, 0].float()


def _plain_logprob(s):
    z, kept, w = _plain_rows(s)
    at = s["ids"].long()[:, None]
    lp = torch.where(kept.gather(1, at), z.gather(1, at) - w.sum(dim=1, keepdim=True).log(), -math.inf)
    return lp[:, 0].float()


def _plain_blocks(s):
    """Growing requests take blocks from the ring in request order; one that the pool cannot serve keeps what it has."""
    mb = s["case"]["max_blocks"]
    more = torch.clamp((s["lens"] + BLOCK - 1) // BLOCK - s["owned"], min=0).long()
    upto = more.cumsum(0)
    more = torch.where(upto <= s["pool"][1], more, 0)
    first = upto - more
    j = torch.arange(mb, device=DEV)[None, :] - s["owned"].long()[:, None]
    fresh = (j >= 0) & (j < more[:, None])
    at = torch.where(fresh, (s["pool"][0] + first[:, None] + j) % s["n_blocks"], 0)
    table = torch.where(fresh, s["ring"][at], s["table"])
    taken = more.sum()
    pool = torch.stack([(s["pool"][0] + taken) % s["n_blocks"], s["pool"][1] - taken]).int()
    return table, (s["owned"] + more).int(), pool


def _plain_slots(s):
    new = s["new"].long()
    row0 = torch.cat([new.new_zeros(1), new.cumsum(0)])
    row = torch.arange(s["rows"], device=DEV)
    used = row < row0[-1]
    seq = torch.clamp(torch.searchsorted(row0[1:], row, right=True), max=len(new) - 1)
    pos = torch.where(used, row - row0[seq] + s["start"][seq], 0)
    slot = s["table"][seq, pos // BLOCK].long() * BLOCK + pos % BLOCK
    return (row0.int(), torch.where(used, seq.int(), s["row_seq"]), torch.where(used, pos.int(), s["row_pos"]),
            torch.where(used, slot, s["slots"]))


# ------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"sample": _plain_sample, "logprob": _plain_logprob, "blocks": _plain_blocks,
                "slots": _plain_slots}[op](state)
    import invariant_forward_policy_gb300 as bi
    c = state["case"]
    if op in ("sample", "logprob"):
        rule = bi.bi_sampling(state["temp"], state["k"], state["p"], state["mp"])
        kind = bi.BI_DTYPE_BF16 if c["dtype"] == "bf16" else bi.BI_DTYPE_FP32
        if op == "sample":
            bi.bi_sample(state["logits"], c["T"], c["V"], rule, state["u"], state["out_ids"], state["out_lp"],
                         dtype=kind, ld=c["V"] + c["pad"])
            return state["out_ids"], state["out_lp"]
        bi.bi_sample_logprob(state["logits"], c["T"], c["V"], rule, state["ids"], state["out_lp"], dtype=kind,
                             ld=c["V"] + c["pad"])
        return state["out_lp"]
    if op == "blocks":
        bi.bi_block_table_resize(state["lens"], c["B"], state["table"], c["max_blocks"], state["owned"],
                                 state["ring"], state["n_blocks"], state["pool"], n_owned_out=state["owned_out"],
                                 pool_out=state["pool_out"])
        return state["table"], state["owned_out"], state["pool_out"]
    bi.bi_slot_map(state["new"], state["start"], c["B"], state["table"], c["max_blocks"], state["n_blocks"],
                   state["rows"], state["row0"], state["row_seq"], state["row_pos"], state["slots"])
    return state["row0"], state["row_seq"], state["row_pos"], state["slots"]


# ------------------------------------------------------------------------------------ 64-bit definitions
def _exact_row(x, temp, k, p, mp):
    """Kept indices (ascending), their masses and scaled logits of one row, by sorting it on the host."""
    if temp == 0:
        temp, k, p, mp = 1.0, 1, 1.0, 0.0
    z = (x - x.max()) / temp
    if k <= 0 and p >= 1:      # no cut that needs an order
        kept = np.flatnonzero(np.exp(z) >= mp) if mp > 0 else np.arange(len(z))
        return kept, np.exp(z[kept]), z[kept]
    order = np.argsort(-x, kind="stable")
    zs = z[order]
    n = len(zs) if k <= 0 else min(int(k), len(zs))
    zs = zs[:n]
    ws = np.exp(zs)
    n = int(np.count_nonzero(ws >= mp)) if mp > 0 else n
    ws = ws[:n]
    if p < 1:
        cum = np.cumsum(ws)
        n = min(n, int(np.searchsorted(cum, p * cum[-1], side="left")) + 1)
    kept = np.sort(order[:n])
    return kept, np.exp(z[kept]), z[kept]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "blocks":
        return _exact_blocks(s)
    if case["op"] == "slots":
        return _exact_slots(s)
    T, V = case["T"], case["V"]
    if T * V > (140_000_000 if case["rule"] in ("temp", "minp") else 40_000_000):
        return None
    x = s["logits"].double().cpu().numpy()[:, :V]
    par = [s[n].cpu().numpy() for n in ("temp", "k", "p", "mp")]
    u = s["u"].double().cpu().numpy()
    ids, lp = np.zeros(T, np.int32), np.zeros(T)
    for t in range(T):
        kept, w, z = _exact_row(x[t], float(par[0][t]), int(par[1][t]), float(par[2][t]), float(par[3][t]))
        cum = np.cumsum(w)
        if case["op"] == "sample":
            j = min(int(np.searchsorted(cum, u[t] * cum[-1], side="right")), len(kept) - 1)
            ids[t] = kept[j]
        else:
            j = int(np.searchsorted(kept, int(s["ids"][t])))
        lp[t] = z[j] - math.log(math.fsum(w))
    return (ids, lp) if case["op"] == "sample" else lp


def _exact_blocks(s):
    table, owned = s["table"].cpu().numpy().copy(), s["owned"].cpu().numpy().copy()
    lens, ring = s["lens"].cpu().numpy(), s["ring"].cpu().numpy()
    head, free = (int(v) for v in s["pool"].cpu())
    room, asked = free, 0
    for b in range(len(lens)):
        need = -(-int(lens[b]) // BLOCK)
        asked += max(0, need - int(owned[b]))
        if asked > room:
            continue
        while owned[b] < need:
            table[b, owned[b]] = ring[head]
            owned[b] += 1
            head, free = (head + 1) % len(ring), free - 1
    return table, owned, np.array([head, free], np.int32)


def _exact_slots(s):
    new, start, table = (s[n].cpu().numpy() for n in ("new", "start", "table"))
    row0, seq, pos, slot = [0], [], [], []
    for b in range(len(new)):
        for i in range(int(new[b])):
            q = int(start[b]) + i
            seq.append(b)
            pos.append(q)
            slot.append(int(table[b, q // BLOCK]) * BLOCK + q % BLOCK)
        row0.append(len(seq))
    rest = [-1] * (s["rows"] - len(seq))
    seq, pos, slot = seq + rest, pos + rest, slot + rest
    return (np.array(row0, np.int32), np.array(seq, np.int32), np.array(pos, np.int32), np.array(slot, np.int64))
