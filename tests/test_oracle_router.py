"""Pins of the router oracle's scored choice (oracle.routing.route_scored):
the plain softmax router as a special case, and a brute-force reading of the
definition on small integers and exact ties."""
import itertools

import numpy as np
import pytest

from oracle import routing as orr


def test_softmax_without_bias_is_the_plain_router():
    z = np.random.default_rng(0).standard_normal((50, 24)).astype(np.float32)
    z[7, 3] = z[7, 11]
    ids, w = orr.route_scored(z, 5)
    ids0, w0 = orr.route_topk(z, 5)
    assert np.array_equal(ids, ids0)
    assert np.array_equal(w.astype(np.float32), w0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_choice_is_the_best_of_all_subsets(score, group_score):
    """Over 8 experts in 4 groups: the chosen pair of groups has the largest
    sum of group values and the chosen experts the largest sum of choice
    values among every subset."""
    rng = np.random.default_rng(1)
    for _ in range(40):
        z = rng.standard_normal((1, 8))
        b = 0.3 * rng.standard_normal(8)
        ids, w = orr.route_scored(z, 3, score, b, 4, 2, group_score, False, 2.5)
        p = np.exp(z[0]) / np.exp(z[0]).sum() if score == "softmax" else 1 / (1 + np.exp(-z[0]))
        c = (p + b).reshape(4, 2)
        v = c.max(1) if group_score == "max" else c.sum(1)
        groups = max(itertools.combinations(range(4), 2), key=lambda g: v[list(g)].sum())
        pool = [2 * g + i for g in groups for i in range(2)]
        best = max(itertools.combinations(pool, 3), key=lambda s: (p + b)[list(s)].sum())
        assert sorted(ids[0]) == sorted(best)
        assert list(ids[0]) == sorted(best, key=lambda e: -(p + b)[e])
        assert np.allclose(w[0], 2.5 * p[ids[0]], rtol=1e-14)


def test_ties_take_the_lower_index():
    z = np.zeros((1, 12), dtype=np.float32)
    for score, b in itertools.product(("softmax", "sigmoid"), (None, np.full(12, 0.25))):
        ids, w = orr.route_scored(z, 4, score, b, 3, 2, "top2")
        assert list(ids[0]) == [0, 1, 2, 3]
        assert np.allclose(w, 0.25)


def test_unavailable_experts():
    inf, nan = np.inf, np.nan
    z = np.array([[1.0, -inf, nan, 0.5], [-inf, nan, -inf, -inf], [inf, 0.0, inf, -inf]])
    ids, w = orr.route_scored(z, 3)
    assert ids.tolist() == [[0, 3, -1], [-1, -1, -1], [0, 2, 1]]
    assert w[1].tolist() == [0, 0, 0] and w[0, 2] == 0 and np.isclose(w[0].sum(), 1)
    assert w[2].tolist() == [0.5, 0.5, 0.0]
    # a bias of -inf or NaN closes an expert to the choice, not to the softmax
    ids, w = orr.route_scored(np.zeros((1, 4)), 2, "softmax", np.array([0.0, -inf, nan, 0.0]), renormalize=False)
    assert ids.tolist() == [[0, 3]] and w.tolist() == [[0.25, 0.25]]
    # a group whose only available expert counts alone
    ids, _ = orr.route_scored(np.array([[2.0, -inf, 0.1, 0.1]]), 1, "sigmoid", None, 2, 1, "top2")
    assert ids.tolist() == [[2]]    # 1/(1+e^-2) = 0.88 < 2 * 0.525
