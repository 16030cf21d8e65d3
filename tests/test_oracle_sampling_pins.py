"""Pins of the sampling oracle against things other than itself: closed forms, torch's softmax,
an enumeration of every prefix, and the frequencies that a fine grid of random numbers gives."""
import math

import numpy as np
import pytest
import torch

from oracle import sampling as osm


def test_temperature_alone_is_a_softmax():
    x = np.random.default_rng(1).standard_normal(200)
    for T in (0.3, 1.0, 2.5):
        want = torch.log_softmax(torch.from_numpy(x) / T, 0).numpy()
        got = [osm.logprob(x, i, temperature=T) for i in range(len(x))]
        assert np.allclose(got, want, rtol=0, atol=1e-12)


def test_draw_frequencies_follow_the_masses():
    # a grid of 2^14 random numbers hits each interval of the running mass in proportion to its length
    x = np.log(np.array([1.0, 5.0, 2.0, 8.0]))
    u = (np.arange(1 << 14) + 0.5) / (1 << 14)
    ids = [osm.draw(x, v)[0] for v in u]
    assert np.allclose(np.bincount(ids, minlength=4) / len(u), np.array([1, 5, 2, 8]) / 16, atol=2.0 / len(u))


def test_draw_borders():
    x = np.zeros(4)
    assert [osm.draw(x, v)[0] for v in (0.0, 0.2499, 0.25, 0.5, 0.75, 0.999)] == [0, 0, 1, 2, 3, 3]


def test_each_cut_by_enumeration():
    rng = np.random.default_rng(3)
    for _ in range(40):
        x = rng.integers(-4, 5, 9) / 2.0      # ties included
        order = sorted(range(9), key=lambda i: (-x[i], i))
        w = np.exp(x - x.max())
        assert osm.kept_tokens(x, top_k=4)[0].tolist() == order[:4]
        p = float(rng.uniform(0.05, 0.99))
        n = min(n for n in range(1, 10) if w[order[:n]].sum() >= p * w.sum() * (1 - 1e-15))
        assert osm.kept_tokens(x, top_p=p)[0].tolist() == order[:n]
        mp = float(rng.uniform(0.01, 0.9))
        assert osm.kept_tokens(x, min_p=mp)[0].tolist() == [i for i in order if w[i] >= mp]


def test_cuts_apply_in_turn():
    x = np.log(np.array([8.0, 4.0, 2.0, 1.0, 1.0]))
    # min-p 0.2 leaves 8, 4, 2; top-k 2 leaves 8, 4; top-p 0.7 of 12 needs both, of 16 only the first two too
    assert osm.kept_tokens(x, min_p=0.2)[0].tolist() == [0, 1, 2]
    assert osm.kept_tokens(x, min_p=0.2, top_k=2, top_p=0.66)[0].tolist() == [0]
    assert osm.kept_tokens(x, top_p=0.66)[0].tolist() == [0, 1]


def test_edges():
    assert osm.draw(np.full(3, -np.inf), 0.5) == (-1, -np.inf)
    assert osm.draw([0.0, 7.0, 7.0], 0.9, temperature=0) == (1, 0.0)
    assert osm.draw([-np.inf, 2.0, -np.inf], 0.99) == (1, 0.0)
    assert osm.kept_tokens([1.0, 2.0, 0.0], top_p=0.0)[0].tolist() == [1]
    assert osm.kept_tokens([1.0, 2.0, 2.0], min_p=1.0)[0].tolist() == [1, 2]
    assert osm.logprob([0.0, 0.0], 1, top_k=1) == -np.inf
    assert osm.logprob([0.0, 0.0], 1) == pytest.approx(-math.log(2), abs=1e-15)
