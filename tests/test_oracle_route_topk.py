"""Pins of the routing oracle: hand values, ties, masks, groups, and its gradient against differences."""

import numpy as np
import pytest

from oracle import route_topk as R
from oracle import router as OR


def test_hand_values():
    l = np.log(np.array([[1.0, 4.0, 3.0, 2.0]]))
    ids, w = R.route(l, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[4 / 7, 3 / 7]], atol=1e-15)
    ids, w = R.route(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [[0.8, 0.6]], atol=1e-15)
    # sigmoid(log a) = a / (1 + a); a bias of 1 on expert 0 brings it to the front, not into its weight
    ids, w = R.route(l, 2, score="sigmoid", bias=np.array([1.0, 0, 0, 0]), renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.5, 0.8]], atol=1e-15)
    ids, w = R.route(l, 2, score="sigmoid", bias=np.array([1.0, 0, 0, 0]))
    assert np.allclose(w, [[0.5 / 1.3, 0.8 / 1.3]], atol=1e-15)


def test_plain_case_is_the_router_step():
    l = np.random.default_rng(0).standard_normal((50, 24))
    ids, w = R.route(l, 5)
    assert np.array_equal(ids, OR.topk_order(l, 5))
    assert np.allclose(w, OR.topk_probs(l, ids), atol=1e-15)


def test_groups():
    l = np.array([[0.0, 5.0, 3.0, 3.5, 4.0, -9.0]])          # groups (0,1) (2,3) (4,5)
    ids, _ = R.route(l, 2, n_group=3, topk_group=1)
    assert ids.tolist() == [[1, 0]]                            # the largest single expert: group 0
    ids, _ = R.route(l, 2, score="sigmoid", n_group=3, topk_group=1, group_score="top2")
    assert ids.tolist() == [[3, 2]]                            # s(3) + s(3.5) > s(0) + s(5)
    ids, _ = R.route(l, 3, n_group=3, topk_group=2)
    assert ids.tolist() == [[1, 4, 0]]


def test_ties_and_masks():
    inf = np.inf
    ids, w = R.route(np.array([[2.0, 2.0, 2.0, 2.0]]), 3)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 3)
    ids, w = R.route(np.array([[-inf, 1.0, np.nan, -inf]]), 3)
    assert ids.tolist() == [[1, 0, 2]] and w.tolist() == [[1.0, 0.0, 0.0]]
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w = R.route(np.full((1, 4), -inf), 2, score=score, renormalize=renorm)
            assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
            assert not R.backward(np.full((1, 4), -inf), ids, np.ones((1, 2)), score, renorm, 1.0).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((6, 10))
    ids, _ = R.route(l, 4, score=score)
    dw = rng.standard_normal((6, 4))
    got = R.backward(l, ids, dw, score, renorm, 1.5)
    h = 1e-5
    for e in range(10):
        up, dn = l.copy(), l.copy()
        up[:, e] += h
        dn[:, e] -= h
        diff = ((R.weights(up, ids, score, renorm, 1.5) - R.weights(dn, ids, score, renorm, 1.5)) * dw).sum(1) / (2 * h)
        # h^2 / 6 times a third derivative of order one, and FP64 rounding over 2h
        assert np.all(np.abs(diff - got[:, e]) <= 1e-9 + 1e-10 * np.abs(got[:, e]))
