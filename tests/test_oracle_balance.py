"""The FP64 balance loss of the oracle: pinned values, the loss of an even router, and its gradient
against differences and against torch's chain rule."""

import numpy as np
import pytest
import torch

from oracle import balance as B


def make(T, E, k, seed=0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((T, E)), np.argsort(-rng.random((T, E)), axis=1)[:, :k].astype(np.int32)


def test_even_router_has_loss_one():
    ids = np.array([[0, 1], [2, 3]], np.int32)
    loss, counts, probs, tokens = B.loss(np.zeros((2, 4)), ids)
    assert np.allclose(loss, [1.0]) and np.array_equal(counts, [[1, 1, 1, 1]]) and np.allclose(probs, 0.25) and tokens == [2]
    # everything on one expert: E times as much
    loss, _, _, _ = B.loss(np.array([[50.0, 0, 0, 0]] * 3), np.zeros((3, 1), np.int32))
    assert np.allclose(loss, [4.0])


def test_by_hand():
    l = np.log(np.array([[1.0, 3.0], [1.0, 1.0]]))                # softmax 1/4, 3/4 and 1/2, 1/2
    ids = np.array([[1], [0]], np.int32)
    loss, counts, probs, tokens = B.loss(l, ids)
    assert np.allclose(probs, [[0.375, 0.625]]) and np.array_equal(counts, [[1, 1]]) and np.allclose(loss, [1.0])
    loss, counts, probs, tokens = B.loss(l, ids, mask=[1, 0])
    assert np.allclose(loss, [2 * 0.75]) and np.array_equal(counts, [[0, 1]]) and tokens == [1]
    # sigmoids 1/2, 3/4 over their sum
    assert np.allclose(B.loss(l, ids, score="sigmoid", mask=[1, 0])[2], [[0.4, 0.6]])


def test_sequences_and_masks():
    l, ids = make(9, 5, 2)
    mask = np.array([1, 1, 0, 1, 0, 0, 1, 1, 1])
    offsets = [1, 4, 4, 6, 8]                                     # rows 0 and 8 belong to none, the second is empty
    loss, counts, probs, tokens = B.loss(l, ids, mask=mask, offsets=offsets)
    assert list(tokens) == [2, 0, 0, 2] and loss[1] == loss[2] == 0 and not probs[1].any() and not counts[2].any()
    one = B.loss(l[[1, 3]], ids[[1, 3]])
    assert np.allclose(loss[0], one[0][0]) and np.array_equal(counts[0], one[1][0])


def test_masked_experts_and_far_logits():
    inf = np.inf
    assert np.array_equal(B.probabilities([-inf, np.nan, -inf], "softmax"), [0, 0, 0])
    assert np.array_equal(B.probabilities([inf, 0.0, inf], "softmax"), [0.5, 0, 0.5])
    assert np.allclose(B.probabilities([-700.0, -701.0], "sigmoid"), B.probabilities([0.0, -1.0], "softmax"))
    assert np.array_equal(B.probabilities([-710.0, -720.0], "sigmoid"), [0, 0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient(score):
    T, E, k = 7, 6, 2
    l, ids = make(T, E, k, 3)
    mask, offsets, dloss = np.array([1, 1, 1, 0, 1, 1, 1]), [0, 4, 6], np.array([0.7, -1.3])
    _, counts, _, tokens = B.loss(l, ids, score, mask, offsets)
    d, _ = B.backward(l, k, counts, tokens, dloss, score, mask, offsets)
    step = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += step
            down[t, e] -= step
            want = (dloss * (B.loss(up, ids, score, mask, offsets)[0] - B.loss(down, ids, score, mask, offsets)[0])).sum() / (2 * step)
            assert abs(d[t, e] - want) < 1e-8
    x = torch.from_numpy(l).requires_grad_(True)
    p = torch.softmax(x, -1) if score == "softmax" else torch.sigmoid(x) / torch.sigmoid(x).sum(-1, keepdim=True)
    total = 0.0
    for s, rows in enumerate(B.members(T, mask, offsets)):
        total = total + dloss[s] * E * (torch.from_numpy(counts[s]).double() * p[rows].mean(0)).sum() / (k * len(rows))
    total.backward()
    assert np.allclose(d, x.grad.numpy(), rtol=0, atol=1e-14)
