"""Pins for oracle.router: hand-worked choices, ties, groups and masks, and the
gradient against central differences of the weights."""

import numpy as np
import pytest

from oracle import router


def test_choice_by_hand():
    l = np.array([0.0, 2.0, 1.0, 2.0])
    assert router.choose(l, 3, "softmax") == [1, 3, 2]                       # the tie goes to the lower id
    assert router.choose(l, 2, "sigmoid", bias=np.array([9.0, 0, 0, 0.1])) == [0, 3]
    l[1] = -np.inf
    assert router.choose(l, 4, "softmax") == [3, 2, 0, 1]                    # off: last
    assert router.choose(l, 2, "sigmoid", bias=np.array([0, 99.0, 0, 0])) == [3, 2]  # whatever its bias


def test_groups_by_hand():
    l = np.array([5.0, -5, 3, 3, 4, 0])
    kw = dict(n_group=3, topk_group=1)
    assert router.choose(l, 1, "sigmoid", group_top=1, **kw) == [0]
    assert router.choose(l, 2, "sigmoid", group_top=2, **kw) == [2, 3]
    l[2:4] = -np.inf
    assert router.choose(l, 2, "sigmoid", group_top=2, **kw) == [4, 5]
    assert router.choose(np.full(6, -np.inf), 2, "softmax", group_top=2, **kw) == [0, 1]


def test_weights_by_hand():
    w, ids = router.route([[0.0, np.log(3.0)]], 2, "softmax", renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[1.5, 0.5]])
    w, _ = router.route([[-np.inf, -np.inf]], 2, "softmax")
    assert w.tolist() == [[0, 0]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_matches_differences(scoring, renorm):
    rng = np.random.default_rng(2)
    l = rng.standard_normal((3, 9))
    l[1, 4] = -np.inf
    _, ids = router.route(l, 4, scoring)
    g = rng.standard_normal((3, 4))
    got = router.route_grad(g, l, ids, scoring, renorm, 2.5)
    f = lambda v, t: (g[t] * router.weights(v, ids[t], scoring, renorm, 2.5)).sum()  # noqa: E731
    for t in range(3):
        for e in range(9):
            if l[t, e] == -np.inf:
                assert got[t, e] == 0
                continue
            d = np.zeros(9)
            d[e] = 1e-5
            # central difference: truncation ~ 1e-10 of third derivatives of order 1, rounding ~ 1e-16 / 1e-5
            assert abs(got[t, e] - (f(l[t] + d, t) - f(l[t] - d, t)) / 2e-5) < 1e-8
