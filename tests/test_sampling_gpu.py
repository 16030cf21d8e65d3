"""bi_sample and bi_sample_logprob on the GPU through the C ABI: tokens equal to the 64-bit oracle's,
logprobs within the fp32 roundings of their formula, the draw's logprob and the score's the same
bits, and rows that do not depend on the batch or on how a row is split."""
import numpy as np
import pytest
import torch

import invariant_forward_policy_gb300 as bi
from oracle import sampling as osm
from tests.gpu_util import same_bits

pytestmark = pytest.mark.gpu


def _rule(T, temp=None, k=None, p=None, mp=None):
    def arr(v, kind):
        return None if v is None else torch.from_numpy(np.broadcast_to(np.asarray(v, kind), (T,)).copy()).cuda()
    return bi.bi_sampling(arr(temp, np.float32), arr(k, np.int32), arr(p, np.float32), arr(mp, np.float32))


def _f32(v):
    return float(np.float32(v))


def _row_rule(t, temp=None, k=None, p=None, mp=None):
    pick = lambda v: np.broadcast_to(np.asarray(v), (t + 1,))[t]  # noqa: E731
    r = {}
    if temp is not None:
        r["temperature"] = _f32(pick(temp))
    if k is not None:
        r["top_k"] = int(pick(k))
    if p is not None:
        r["top_p"] = _f32(pick(p))
    if mp is not None:
        r["min_p"] = _f32(pick(mp))
    return r


def _padded(x, ld, dtype):
    """x [T, V] in rows of ld elements, the rest NaN (which nothing may read)."""
    T, V = x.shape
    full = torch.full((T, ld), float("nan"), dtype=dtype, device="cuda")
    full[:, :V] = x.to(dtype)
    return full


def _run(x, u, dtype=torch.float32, ld=None, **rule):
    """x fp32 host [T, V] -> (ids, lp) of the draw, checked to be the score's bits, and the values as stored."""
    T, V = x.shape
    ld = V if ld is None else ld
    dev = _padded(torch.from_numpy(x).cuda(), ld, dtype)
    kind = bi.BI_DTYPE_BF16 if dtype == torch.bfloat16 else bi.BI_DTYPE_FP32
    sp = _rule(T, **rule)
    ids = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((T,), float("nan"), device="cuda")
    bi.bi_sample(dev, T, V, sp, torch.from_numpy(np.asarray(u, np.float32)).cuda(), ids, lp, dtype=kind, ld=ld)
    lp2 = torch.full((T,), float("nan"), device="cuda")
    bi.bi_sample_logprob(dev, T, V, sp, torch.clamp(ids, min=0), lp2, dtype=kind, ld=ld)
    torch.cuda.synchronize()
    assert same_bits(lp, lp2)
    return ids.cpu().numpy(), lp.cpu().numpy(), dev[:, :V].float().cpu().numpy()


def _tol(z, lp):
    """The logprob is (x - m)/T - e ln2 - ln(mant): the two-float product's high part enters a fused multiply-add
    and two sums, each rounded at 2^-24 of a term no larger than |z| + |lp| + 1; logf's error is within 2^-23 of
    at most 0.41.  The masses (5e-10 each, cut at 2^-56 of the largest: 2^18 of them at most) add 1e-8."""
    return 2.0 ** -24 * (3 * (np.abs(z) + np.abs(lp) + 1) + 1) + 1e-8


def _check(x, u, ids, lp, **rule):
    for t in range(len(x)):
        r = _row_rule(t, **rule)
        want, wlp = osm.draw(x[t], _f32(u[t]), **r)
        assert ids[t] == want, (t, r, u[t], ids[t], want)
        if want < 0:
            assert lp[t] == -np.inf
            continue
        z = (float(x[t, want]) - float(x[t].max())) / (r.get("temperature", 1.0) or 1.0)
        assert abs(float(lp[t]) - wlp) <= _tol(z, wlp), (t, r, float(lp[t]), wlp)


def _logits(rng, T, V, dist):
    if dist == "flat":
        return rng.standard_normal((T, V)).astype(np.float32)
    if dist == "peaked":
        x = (2.5 * rng.standard_normal((T, V))).astype(np.float32)
        at = rng.integers(0, V, (T, 12))
        x[np.arange(T)[:, None], at] = rng.uniform(3, 18, (T, 12))
        return x
    if dist == "coarse":      # a handful of values: ties everywhere, both zeros, masked places
        x = rng.integers(-3, 3, (T, V)).astype(np.float32)
        zero = x == 0
        x[zero] = np.where(rng.random(zero.sum()) < 0.5, np.float32(0.0), np.float32(-0.0))
        x[rng.random((T, V)) < 0.2] = -np.inf
        x[:, 0] = 2.0
        return x
    assert dist == "wide"     # large, offset and far apart
    return (1000.0 + 40.0 * rng.standard_normal((T, V))).astype(np.float32)


RULES = {
    "plain": dict(),
    "temp": dict(temp=0.7),
    "topk": dict(temp=1.3, k=7),
    "topk_large": dict(k=1500),
    "topp": dict(temp=0.9, p=0.9),
    "topp_tight": dict(p=0.05),
    "minp": dict(mp=0.03),
    "topk_topp": dict(temp=0.8, k=40, p=0.95),
    "topk_large_topp": dict(k=1100, p=0.8),
    "all": dict(temp=1.1, k=60, p=0.97, mp=0.01),
}


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("dist", ["flat", "peaked", "coarse", "wide"])
@pytest.mark.parametrize("T,V,ld,dtype", [(5, 2500, 2500, torch.float32), (3, 5003, 5006, torch.bfloat16),
                                          (2, 40001, 40001, torch.float32)])
def test_draw_and_score_match_the_oracle(rule, dist, T, V, ld, dtype):
    rng = np.random.default_rng([T, V, len(rule), len(dist)])
    u = rng.random(T).astype(np.float32)
    ids, lp, x = _run(_logits(rng, T, V, dist), u, dtype, ld, **RULES[rule])
    _check(x, u, ids, lp, **RULES[rule])
    assert bi.bi_device_status() == 0


@pytest.mark.parametrize("V", [1, 2, 3, 7, 31, 127, 128, 129, 1023, 1025, 4096])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_and_odd_vocabularies(V, dtype):
    rng = np.random.default_rng(V)
    T = 6
    u = np.array([0.0, 2.0 ** -24, 1e-30, 0.5, 0.7, 1 - 2.0 ** -24], np.float32)
    for pad in (0, 1, 5):
        for rule in (dict(), dict(k=3), dict(p=0.6), dict(temp=0.5, k=2, p=0.5, mp=0.2)):
            ids, lp, x = _run(_logits(rng, T, V, "flat"), u, dtype, V + pad, **rule)
            _check(x, u, ids, lp, **rule)
    assert bi.bi_device_status() == 0


@pytest.mark.parametrize("V", [3000, 70000, 262144])
@pytest.mark.parametrize("rule", [dict(), dict(k=5), dict(k=2000), dict(p=0.5), dict(k=2900, p=0.25),
                                  dict(temp=0.0)])
def test_equal_logits(V, rule):
    """Every logit the same: the cut counts ties out by index, beyond what the sort holds."""
    x = np.full((3, V), -3.25, np.float32)
    u = np.array([0.0, 0.5, 1 - 2.0 ** -24], np.float32)
    ids, lp, _ = _run(x, u, **rule)
    kept = V
    if rule.get("temp") == 0.0:
        kept = 1
    if "k" in rule:
        kept = min(kept, rule["k"])
    if "p" in rule:
        kept = -(-kept * int(rule["p"] * 4) // 4)
    assert ids.tolist() == [0, kept // 2, int(np.floor(float(u[2]) * kept))]
    assert np.all(np.abs(lp + np.log(kept)) <= _tol(0.0, np.log(kept)))


@pytest.mark.parametrize("rule", [dict(), dict(p=0.9), dict(k=3000), dict(k=1500, p=0.7), dict(k=10)])
def test_many_ties_at_the_cut(rule):
    """Few distinct values over a large row: bins and equal-value groups larger than the sort holds."""
    rng = np.random.default_rng(11)
    V, T = 60000, 4
    x = rng.choice(np.array([-1.0, -1.0 + 2.0 ** -20, 0.5, 0.5 + 2.0 ** -22, 3.0], np.float32), (T, V),
                   p=[0.3, 0.3, 0.2, 0.1999, 0.0001])
    u = rng.random(T).astype(np.float32)
    ids, lp, x = _run(x, u, **rule)
    _check(x, u, ids, lp, **rule)


@pytest.mark.parametrize("temp", [2.0 ** -60, 1e-6, 1e-3, 0.02, 50.0, 1e9])
def test_extreme_temperatures(temp):
    rng = np.random.default_rng(5)
    for rule in (dict(temp=temp), dict(temp=temp, k=30), dict(temp=temp, p=0.9), dict(temp=temp, k=1200, p=0.9),
                 dict(temp=temp, mp=0.1)):
        x = _logits(rng, 3, 9000, "peaked")
        u = rng.random(3).astype(np.float32)
        ids, lp, x = _run(x, u, **rule)
        _check(x, u, ids, lp, **rule)


def test_top_k_reaches_tokens_without_mass():
    """At a low temperature the k-th token lies far below the masses: the score still tells kept from cut."""
    V, k = 5000, 1500
    x = np.sort(np.random.default_rng(8).standard_normal(V).astype(np.float32))[::-1][None].copy()
    dev = torch.from_numpy(np.repeat(x, 4, 0)).cuda()
    ids = torch.tensor([0, k - 1, k, V - 1], dtype=torch.int32, device="cuda")
    for kk in (k, 700):
        ids[1], ids[2] = kk - 1, kk
        lp = torch.empty(4, device="cuda")
        bi.bi_sample_logprob(dev, 4, V, _rule(4, temp=0.01, k=kk), ids, lp)
        got = lp.cpu().numpy()
        want = [osm.logprob(x[0], int(i), temperature=_f32(0.01), top_k=kk) for i in ids.cpu()]
        assert got[2] == got[3] == -np.inf and want[2] == want[3] == -np.inf
        for g, w in zip(got[:2], want[:2]):
            assert abs(g - w) <= _tol(w, w)


def test_masked_rows_and_lowest_values():
    V = 6000
    x = np.full((6, V), -np.inf, np.float32)
    x[1, 4321] = -2.0                                  # one token left
    x[2] = np.finfo(np.float32).min                    # every logit the type's lowest value
    x[3] = np.finfo(np.float32).min
    x[3, 17] = 0.0
    x[4, ::7] = np.random.default_rng(2).standard_normal(len(x[4, ::7]))
    x[5, -1] = np.finfo(np.float32).max
    x[5, 0] = np.finfo(np.float32).min
    u = np.full(6, 0.6, np.float32)
    for rule in (dict(), dict(k=5), dict(p=0.9), dict(k=2500, p=0.9), dict(mp=0.5), dict(temp=0.0)):
        ids, lp, _ = _run(x, u, **rule)
        _check(x, u, ids, lp, **rule)
    assert ids[0] == -1 and lp[0] == -np.inf
    assert bi.bi_device_status() == 0                  # a row with nothing left is no error


def test_refused_rows_leave_the_others():
    rng = np.random.default_rng(4)
    T, V = 8, 3100
    x = _logits(rng, T, V, "flat")
    x[1, 700] = np.nan
    x[3, 5] = np.inf
    u = rng.random(T).astype(np.float32)
    u[5] = 1.0
    p = np.ones(T, np.float32)
    p[6] = np.nan
    temp = np.ones(T, np.float32)
    temp[7] = -0.5
    dev = torch.from_numpy(x).cuda()
    ids = torch.full((T,), -9, dtype=torch.int32, device="cuda")
    lp = torch.zeros(T, device="cuda")
    bi.bi_sample(dev, T, V, _rule(T, temp=temp, p=p), torch.from_numpy(u).cuda(), ids, lp)
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    assert bi.bi_device_status() == 0                  # cleared
    got, glp = ids.cpu().numpy(), lp.cpu().numpy()
    for t in range(T):
        if t in (1, 3, 5, 6, 7):
            assert got[t] == -1 and np.isnan(glp[t])
        else:
            want, wlp = osm.draw(x[t], _f32(u[t]))
            assert got[t] == want and abs(glp[t] - wlp) <= _tol(0, wlp) + 2.0 ** -20
    # a token outside the vocabulary, a parameter row outside the table
    sc = torch.zeros(2, device="cuda")
    bi.bi_sample_logprob(dev, 2, V, None, torch.tensor([V, 3], dtype=torch.int32, device="cuda"), sc)
    assert np.isnan(sc[0].item())
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK
    one = bi.bi_sampling(torch.ones(1, device="cuda"))
    bi.bi_sample(dev, 1, V, one, torch.zeros(1, device="cuda"), ids, lp,
                 param_row=torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert ids[0].item() == -1 and bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK


@pytest.mark.parametrize("V", [3000, 30000, 129280])
def test_rows_do_not_depend_on_the_batch(V):
    """A row alone (split over a cluster) and in a batch that fills the GPU (another split) give the same bits."""
    rng = np.random.default_rng(V)
    T = 320
    x = torch.from_numpy(_logits(rng, 4, V, "peaked")).cuda().repeat(T // 4, 1)
    u = torch.from_numpy(rng.random(T).astype(np.float32)).cuda()
    kw = dict(temp=rng.uniform(0.5, 1.5, T), k=rng.choice([0, 3, 50, 1800], T), p=rng.choice([1.0, 0.9, 0.99], T),
              mp=rng.choice([0.0, 0.02], T))
    sp = _rule(T, **kw)
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    lp = torch.empty(T, device="cuda")
    bi.bi_sample(x, T, V, sp, u, ids, lp)
    i1 = torch.empty(1, dtype=torch.int32, device="cuda")
    l1 = torch.empty(1, device="cuda")
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    for t in list(range(12)) + [T - 1]:
        bi.bi_sample(x[t], 1, V, sp, u[t:t + 1], i1, l1, param_row=rows[t:t + 1])
        assert i1.item() == ids[t].item() and same_bits(l1, lp[t:t + 1])
    perm = torch.randperm(T, device="cuda")
    ids2, lp2 = torch.empty_like(ids), torch.empty_like(lp)
    bi.bi_sample(x[perm].contiguous(), T, V, sp, u[perm].contiguous(), ids2, lp2, param_row=rows[perm].contiguous())
    assert torch.equal(ids2, ids[perm]) and same_bits(lp2, lp[perm])


def test_parameter_rows_and_optional_outputs():
    rng = np.random.default_rng(9)
    T, V = 7, 2000
    x = torch.from_numpy(_logits(rng, T, V, "peaked")).cuda()
    u = torch.from_numpy(rng.random(T).astype(np.float32)).cuda()
    sp = bi.bi_sampling(temperature=torch.tensor([0.5, 1.5], device="cuda"),
                        top_k=torch.tensor([3, 0], dtype=torch.int32, device="cuda"))
    pr = torch.tensor([0, 1, 1, 0, 0, 1, 0], dtype=torch.int32, device="cuda")
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    bi.bi_sample(x, T, V, sp, u, ids, param_row=pr)      # no logprob wanted
    for t in range(T):
        r = [dict(temperature=0.5, top_k=3), dict(temperature=1.5)][int(pr[t])]
        assert ids[t].item() == osm.draw(x[t].cpu().numpy(), u[t].item(), **r)[0]


def test_a_captured_step_walks_its_random_numbers():
    """One graph, replayed with a step counter that selects the row of u; on a stream of its own."""
    rng = np.random.default_rng(10)
    T, V, steps = 3, 8192, 5
    x = torch.from_numpy(_logits(rng, T, V, "peaked")).cuda()
    u = torch.from_numpy(rng.random((steps, T)).astype(np.float32)).cuda()
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    lp = torch.empty(T, device="cuda")
    sp = _rule(T, temp=0.9, k=50, p=0.95)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        bi.bi_sample(x, T, V, sp, u, ids, lp, u_rows=steps, u_row=step)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            bi.bi_sample(x, T, V, sp, u, ids, lp, u_rows=steps, u_row=step)
        for s in range(steps):
            step.fill_(s)
            g.replay()
            st.synchronize()
            for t in range(T):
                want, _ = osm.draw(x[t].cpu().numpy(), u[s, t].item(), temperature=_f32(0.9), top_k=50,
                                   top_p=_f32(0.95))
                assert ids[t].item() == want
        step.fill_(steps)                                # beyond the rows of u: refused
        g.replay()
        st.synchronize()
    assert ids.cpu().tolist() == [-1] * T
    assert bi.bi_device_status() == bi.BI_ERR_DEVICE_CHECK


@pytest.mark.parametrize("T,V,ld,dtype", [(3, 129280, 129280, torch.float32), (3, 262144, 262147, torch.bfloat16),
                                          (160, 129280, 129281, torch.bfloat16), (310, 70001, 70001, torch.float32)])
@pytest.mark.parametrize("dist", ["flat", "peaked"])
def test_long_rows_match_the_oracle(T, V, ld, dtype, dist):
    """Every split of a row, long rows, and the rules side by side in one call; the oracle on a few of the rows."""
    rng = np.random.default_rng([T, V, len(dist)])
    x = np.tile(_logits(rng, 8, V, dist), (-(-T // 8), 1))[:T]
    u = rng.random(T).astype(np.float32)
    rule = dict(temp=rng.uniform(0.6, 1.2, T), k=rng.choice([0, 1, 50, 300, 700, 1024, 1025, 20000, V, V + 1], T),
                p=rng.choice([-1.0, 0.0, 0.5, 0.9, 0.999, 1.0, 2.0], T), mp=rng.choice([-1.0, 0.0, 1e-4, 0.05, 1.0], T))
    ids, lp, stored = _run(x, u, dtype, ld, **rule)
    for t in rng.choice(T, min(T, 24), replace=False):
        one = slice(t, t + 1)
        _check(stored[one], u[one], ids[one], lp[one], **{k: v[t] for k, v in rule.items()})
    assert bi.bi_device_status() == 0


def test_calls_on_two_streams_at_once():
    """Nothing is shared between calls: two streams, each its own rows, interleaved."""
    rng = np.random.default_rng(12)
    T, V = 40, 33000
    rule = dict(temp=0.8, k=rng.choice([0, 50, 2000], T), p=rng.choice([0.9, 1.0], T))
    sp = _rule(T, **rule)
    sides = []
    for _ in range(2):
        x = torch.from_numpy(_logits(rng, T, V, "peaked")).cuda()
        u = torch.from_numpy(rng.random(T).astype(np.float32)).cuda()
        ids = torch.empty((8, T), dtype=torch.int32, device="cuda")
        sides.append((x, u, ids, torch.empty((8, T), device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for k in range(8):
        for x, u, ids, lp, st in sides:
            bi.bi_sample(x, T, V, sp, u, ids[k], lp[k], stream=st)
    torch.cuda.synchronize()
    for x, u, ids, lp, _ in sides:
        want, wlp = torch.empty_like(ids[0]), torch.empty_like(lp[0])
        bi.bi_sample(x, T, V, sp, u, want, wlp)
        for k in range(8):
            assert torch.equal(ids[k], want) and same_bits(lp[k], wlp)
    assert bi.bi_device_status() == 0


@pytest.mark.parametrize("rule", ["temp", "topk", "topk_large", "topp", "minp", "topk_topp"])
@pytest.mark.parametrize("V", [1, 2, 35, 2031, 40001])
def test_zero_draws_the_first_token_of_any_mass(rule, V):
    """u = 0: masses far below the fixed-point unit count, those that 64 bits do not hold do not; the next u after
    it, on rows with nothing so small, is the first token too."""
    rng = np.random.default_rng([V, len(rule)])
    T = 6
    x = (300.0 * rng.standard_normal((T, V))).astype(np.float32)
    x[:, 0] = x.max(1) - np.float32([0.0, 30.0, 60.0, 200.0, 3000.0, np.inf])   # of the largest's mass, or of none
    r = dict(RULES[rule])
    u = np.zeros(T, np.float32)
    ids, lp, st = _run(x, u, **r)
    _check(st, u, ids, lp, **r)
    x = rng.standard_normal((T, V)).astype(np.float32)
    u[:] = 2.0 ** -40
    ids, lp, st = _run(x, u, **r)
    _check(st, u, ids, lp, **r)
    assert bi.bi_device_status() == 0
