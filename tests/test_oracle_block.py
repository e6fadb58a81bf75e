"""Pins of the oracle's dense product, group-limited routing and norms between blocks: closed forms, brute force, and the
library's own elementary functions."""

import itertools
import math

import numpy as np
import pytest

from oracle import linear as ol, prompt, routing


def test_linear_matches_sums_of_products():
    rng = np.random.default_rng(1)
    x, w, b, r = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=4), rng.normal(size=(3, 4))
    f = {None: lambda z: z, "relu": lambda z: max(z, 0.0), "silu": lambda z: z / (1 + math.exp(-z)),
         "gelu": lambda z: 0.5 * z * (1 + math.erf(z / math.sqrt(2))), "sigmoid": lambda z: 1 / (1 + math.exp(-z))}
    for act, fn in f.items():
        y, tol = ol.linear(x, w, b, act, r)
        for m, n in itertools.product(range(3), range(4)):
            z = math.fsum(x[m, k] * w[n, k] for k in range(5)) + b[n]
            assert abs(y[m, n] - (fn(z) + r[m, n])) < 1e-14
        assert (tol > 0).all() and (tol < 1e-4).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,group_top,k", [(8, 4, 2, 2, 3), (9, 3, 1, 1, 2), (6, 1, 1, 1, 4), (6, 6, 4, 1, 3)])
def test_route_groups_by_brute_force(score, bias, E, groups, top_groups, group_top, k):
    rng = np.random.default_rng(E)
    l = rng.normal(size=(20, E))
    b = 0.3 * rng.normal(size=E) if bias else None
    ids, w, gaps = routing.route_groups(l, b, k, score, groups, top_groups, group_top, True, 2.0)
    raw = routing.route_groups(l, b, k, score, groups, top_groups, group_top, False, 2.0)[1]
    assert (gaps > 0).all()
    for t in range(20):
        p = np.exp(l[t]) / np.exp(l[t]).sum() if score == "softmax" else 1 / (1 + np.exp(-l[t]))
        key = p + b if bias else p
        # Without a bias and with one key a group, a group's rank by score is its rank by logit.
        size = E // groups
        worth = [np.sort(key[g * size:(g + 1) * size])[-group_top:].sum() for g in range(groups)]
        best = max(itertools.combinations(range(groups), top_groups), key=lambda c: sum(worth[g] for g in c))
        left = [e for e in range(E) if e // size in best]
        picks = max(itertools.permutations(left, k), key=lambda c: [key[e] for e in c])
        assert ids[t].tolist() == list(picks)
        assert np.allclose(w[t], 2 * p[list(picks)] / p[list(picks)].sum()) and np.allclose(raw[t], 2 * p[list(picks)])


def test_route_groups_without_limits_is_the_routing_rule():
    rng = np.random.default_rng(2)
    l, b = rng.normal(size=(30, 40)).astype(np.float32), (0.1 * rng.normal(size=40)).astype(np.float32)
    ids, w, _ = routing.route(l, b, 5, 2.5)
    got = routing.route_groups(l, b, 5, scale=2.5)
    assert np.array_equal(got[0], ids) and np.allclose(got[1], w, rtol=1e-6)


def test_route_groups_of_nothing():
    l = np.full((1, 8), -np.inf)
    for score in ("sigmoid", "softmax"):
        ids, w, _ = routing.route_groups(l, None, 3, score, 4, 2, 2)
        assert ids[0].tolist() == [0, 1, 2] and not w.any()


def test_block_norm_parts():
    rng = np.random.default_rng(3)
    T, H, k = 4, 16, 3
    x, r, sh = rng.normal(size=(T * k, H)), rng.normal(size=(T, H)), rng.normal(size=(T, H))
    w, pg, g, gate = rng.uniform(size=(T, k)), rng.normal(size=H), rng.normal(size=H), rng.normal(size=(T, H))
    h, y, dh, dy = prompt.block_norm(x, g, r, w, sh, pg, gate, 0.5, 1e-5)
    for t in range(T):
        o = [math.fsum([w[t, j] * x[t * k + j, i] for j in range(k)] + [sh[t, i]]) for i in range(H)]
        rms = math.sqrt(math.fsum(v * v for v in o) / H + 1e-5)
        hh = [0.5 * r[t, i] + gate[t, i] * o[i] / rms * pg[i] for i in range(H)]
        rms = math.sqrt(math.fsum(v * v for v in hh) / H + 1e-5)
        assert np.allclose(h[t], hh, rtol=1e-13) and np.allclose(y[t], [hh[i] / rms * g[i] for i in range(H)], rtol=1e-13)
    assert (dh > 0).all() and (dy > 0).all() and dy.max() < 1e-4
    # Without post norm, gate and routes it is the residual norm.
    x, r = (np.round(v[:T] * 256) / 256 for v in (x, r))  # BF16 sums without rounding are not asked for here
    h, y, _, _ = prompt.block_norm(x, g, r)
    assert np.allclose(h, x + r, rtol=1e-15)
    z = x + r
    assert np.allclose(y, z / np.sqrt((z * z).mean(1, keepdims=True) + 1e-5) * g, rtol=1e-13)
    assert not prompt.block_norm(np.zeros((2, 8)), np.ones(8), post_gamma=np.ones(8))[1].any()
