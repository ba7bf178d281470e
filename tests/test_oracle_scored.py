"""Pins of the scored router's oracle and of the int8 row quantisation's."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle import numerics as nx

LOW = oracle.moe.LOWEST_BF16


def _logits(B, E, seed):
    return np.random.default_rng(seed).standard_normal((B, E)).astype(np.float32)


def test_agrees_with_route_where_the_rules_coincide():
    lg = _logits(64, 24, 1)
    ids, gates = oracle.route(lg, 5)
    got, w = oracle.route_scored(lg, 5, "softmax")
    np.testing.assert_array_equal(got, ids)
    np.testing.assert_allclose(w, gates, rtol=1e-12)
    # sigmoid is monotone: the same picks
    np.testing.assert_array_equal(oracle.route_scored(lg, 5, "sigmoid")[0], ids)


def test_softmax_without_renormalisation_is_the_full_softmax():
    lg = _logits(8, 12, 2)
    ids, w = oracle.route_scored(lg, 12, "softmax", renorm=False, scale=2.5)
    p = np.exp(lg.astype(np.float64))
    p /= p.sum(1, keepdims=True)
    np.testing.assert_allclose(w, 2.5 * np.take_along_axis(p, ids.astype(np.int64), 1), rtol=1e-12)
    np.testing.assert_allclose(w.sum(1), 2.5, rtol=1e-12)


def test_groups_by_hand():
    # sigmoid(0) = 0.5; scores by bias alone
    lg = np.zeros((1, 8), np.float32)
    bias = np.array([0.4, 0.0, 0.3, 0.2, 0.0, 0.1, 0.25, 0.26])
    # sums of the two best: 0.4, 0.5, 0.1, 0.51 (+ 1): groups 3 and 1
    ids, w = oracle.route_scored(lg, 3, "sigmoid", bias, n_groups=4, topk_groups=2, group_top=2)
    np.testing.assert_array_equal(ids, [[2, 7, 6]])
    np.testing.assert_allclose(w, [[1 / 3] * 3])
    # best alone: 0.4, 0.3, 0.1, 0.26: groups 0 and 1
    ids, _ = oracle.route_scored(lg, 3, "sigmoid", bias, n_groups=4, topk_groups=2, group_top=1)
    np.testing.assert_array_equal(ids, [[0, 2, 3]])


def test_ties_go_to_the_lower_group_and_id():
    lg = np.zeros((1, 12), np.float32)
    ids, _ = oracle.route_scored(lg, 4, "sigmoid", n_groups=4, topk_groups=2)
    np.testing.assert_array_equal(ids, [[0, 1, 2, 3]])


def test_masks():
    lg = np.zeros((3, 6), np.float32)
    lg[0, 1:] = -np.inf                       # one expert left
    lg[1] = LOW                               # none left
    lg[2, :2] = np.finfo(np.float32).min      # group 0 is out
    ids, w = oracle.route_scored(lg, 2, "softmax", n_groups=3, topk_groups=1, group_top=2)
    np.testing.assert_array_equal(ids, [[0, -1], [-1, -1], [2, 3]])
    np.testing.assert_allclose(w, [[1, 0], [0, 0], [0.5, 0.5]])
    # a masked bias takes the expert out of the choice, not out of the softmax
    bias = np.zeros(6)
    bias[0] = -np.inf
    ids, w = oracle.route_scored(np.zeros((1, 6), np.float32), 2, "softmax", bias, renorm=False)
    np.testing.assert_array_equal(ids, [[1, 2]])
    np.testing.assert_allclose(w, [[1 / 6, 1 / 6]])
    # a group with one expert left counts that one: 1.1 against 0.5 + 0.55
    lg = np.zeros((1, 4), np.float32)
    lg[0, 1] = -np.inf
    bias = np.array([0.6, 0.0, 0.0, 0.05])
    ids, _ = oracle.route_scored(lg, 2, "sigmoid", bias, n_groups=2, topk_groups=1, group_top=2)
    np.testing.assert_array_equal(ids, [[0, -1]])


def test_nan_ranks_last_and_reaches_its_weight():
    lg = np.zeros((1, 4), np.float32)
    lg[0, 0] = np.nan
    ids, w = oracle.route_scored(lg, 3, "sigmoid", renorm=False)
    np.testing.assert_array_equal(ids, [[1, 2, 3]])
    ids, w = oracle.route_scored(lg, 4, "sigmoid", renorm=False)
    np.testing.assert_array_equal(ids, [[1, 2, 3, 0]])
    assert np.isnan(w[0, 3]) and np.all(w[0, :3] == 0.5)


@pytest.mark.parametrize("seed", range(6))
def test_ranking_by_counting(seed):
    """The picks are the experts that fewer than K others of kept groups beat,
    where a kept group is one that fewer than topk_groups others beat."""
    rng = np.random.default_rng(seed)
    G, S, K, keep, top = 4, 5, 6, 2, 1 + seed % 2
    E = G * S
    lg = rng.integers(-2, 3, (32, E)).astype(np.float32)
    bias = rng.integers(-1, 2, E) * 0.125
    ids, _ = oracle.route_scored(lg, K, "sigmoid", bias, G, keep, top)
    for t in range(32):
        c = 1 / (1 + np.exp(-lg[t].astype(np.float64))) + bias
        gs = [sum(sorted(c[g * S:(g + 1) * S])[::-1][:top]) for g in range(G)]
        kept = [g for g in range(G) if sum((gs[h] > gs[g]) or (gs[h] == gs[g] and h < g) for h in range(G)) < keep]
        on = [e for e in range(E) if e // S in kept]
        rank = {e: sum((c[f] > c[e]) or (c[f] == c[e] and f < e) for f in on) for e in on}
        want = sorted((e for e in on if rank[e] < K), key=lambda e: rank[e])
        np.testing.assert_array_equal(ids[t], want)


# ---------------------------------------------------------------------------- int8 rows
def _exact_code(v, s):
    """Nearest integer to v / s, ties to even, by rational arithmetic."""
    q = Fraction(float(v)) / Fraction(float(s))
    n = q.numerator // q.denominator
    r = q - n
    return n + (1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and n % 2) else 0)


@pytest.mark.parametrize("bf16", [False, True])
def test_int8_rows_against_rational_arithmetic(bf16):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((24, 80)) * np.exp(rng.standard_normal((24, 1)) * 8)).astype(np.float32)
    x[3] = 0.0
    x[4] = 0.0
    x[4, 7] = 127.0                                   # scale 1: half-integers are ties
    x[4, 8:20] = np.arange(12) + 0.5
    x[5] *= np.float32(1e-38)                         # subnormal values, scale at its floor
    x[6, 0] = np.float32(3.3e38)                      # still finite in bf16
    if bf16:
        x = nx.to_bf16(x).astype(np.float32)
    q, s = nx.quantize_i8_rows(x)
    assert q.dtype == np.int8 and s.dtype == np.float32
    for r in range(24):
        a = Fraction(float(np.max(np.abs(x[r]))))
        want = 1.0 if a == 0 else max(np.float32(float(a / 127)), np.float32(2.0**-126))
        assert s[r] == np.float32(want)
        assert [int(v) for v in q[r]] == [_exact_code(v, s[r]) for v in x[r]]
    assert np.abs(q.astype(int)).max() == 127
    np.testing.assert_array_equal(q[4, 8:20], np.rint(np.arange(12) + 0.5))


def test_int8_rows_with_values_that_are_not_finite():
    x = np.ones((3, 16), np.float32)
    x[0, 3], x[1, 4] = np.nan, -np.inf
    q, s = nx.quantize_i8_rows(x)
    assert np.isnan(s[:2]).all() and not q[:2].any()
    assert s[2] == np.float32(1 / 127) and (q[2] == 127).all()
