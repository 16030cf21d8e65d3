"""Token sampling oracle (test infrastructure only): one row at a time, in 64 bits.

[Article] §2 asks that discrete choices and logprobs be the row's own.  The definition is the
library's: masses w_i = exp((x_i - max x) / T), tokens ordered by (logit descending, index
ascending), a kept prefix cut by min-p, then top-k, then top-p, and the draw in index order.
Nothing here is blocked, binned or fixed-point.  A token whose mass rounds to 0 in 64 bits is kept or cut by
its place in the order like any other, has the formula's logprob when kept, and is drawn by no u.

[Article] is "vLLM Achieves Bitwise-Consistent RL Training: Eliminating Numerical
Drift to Zero KL Divergence on DeepSeek-V4-Flash at 91% Throughput"; section numbers
are its own.
"""
from __future__ import annotations

import math

import numpy as np


def kept_tokens(x, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Indices of the kept tokens of one row, in kept order, and every token's scaled logit."""
    x = np.asarray(x, np.float64)
    if not (x > -np.inf).any():
        return np.zeros(0, np.int64), x
    if temperature == 0:
        temperature, top_k, top_p, min_p = 1.0, 1, 1.0, 0.0
    z = (x - x.max()) / float(temperature)
    order = [int(i) for i in np.lexsort((np.arange(len(x)), -x)) if x[i] > -np.inf]
    if min_p >= 1:
        order = [i for i in order if z[i] == 0]
    elif min_p > 0:
        order = [i for i in order if math.exp(z[i]) >= float(min_p)]
    if 0 < top_k < len(order):
        order = order[:top_k]
    if top_p < 1:
        w = np.exp(z[order])
        cum = np.cumsum(w)
        need = max(float(top_p), 0.0) * cum[-1]
        n = 1
        while n < len(order) and cum[n - 1] < need:
            n += 1
        order = order[:n]
    return np.array(order, np.int64), z


def draw(x, u, **rule):
    """(token, logprob) of one row for a random number u in [0, 1)."""
    kept, z = kept_tokens(x, **rule)
    if not len(kept):
        return -1, -np.inf
    kept = np.sort(kept)
    w = np.exp(z[kept])
    total = math.fsum(w)
    run = np.cumsum(w)
    j = int(np.argmax(run > float(u) * run[-1]))
    return int(kept[j]), float(z[kept[j]] - math.log(total))


def logprob(x, token, **rule):
    """Logprob of a given token under the same distribution (-inf when it is cut off)."""
    kept, z = kept_tokens(x, **rule)
    if token not in set(kept.tolist()):
        return -np.inf
    return float(z[token] - math.log(math.fsum(np.exp(z[kept]))))
