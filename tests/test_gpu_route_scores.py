"""The scores that moe_route_topk orders the experts by are the FP32 scores its weights are made of.

With a bias of zero the order value of an expert is its score, so the weights that come back (not renormalised,
scale 1: the scores themselves) descend, and equal ones stand in the order of their ids, bit for bit: there is no
tolerance.  Logits that are close together show any other arithmetic."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import route_topk as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def close_logits(T, E, centre, seed):
    """Rows of logits a few units in the last place of 1 apart."""
    g = torch.Generator().manual_seed(seed)
    steps = torch.randint(-64, 65, (T, E), generator=g).float() * 2.0 ** -23
    return (centre + steps).cuda()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 8), (64, 16), (128, 32), (250, 32), (512, 32), (1024, 32)])
@pytest.mark.parametrize("centre", [0.0, 0.5, -0.7, 1.3, -2.0])
def test_order_is_that_of_the_scores(score, E, k, centre):
    l = close_logits(200, E, centre, seed=E)
    bias = torch.zeros(E, device="cuda")
    ids, w = M.moe_route_topk(l, k, score=score, bias=bias, renormalize=False)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert np.all(w[:, 1:] <= w[:, :-1])
    tie = w[:, 1:] == w[:, :-1]
    assert np.all(ids[:, 1:][tie] > ids[:, :-1][tie])
    # and what was not chosen does not come before: all the scores of a row, from the weights of single experts
    if E == 64:
        s = np.empty((200, E), np.float32)
        for e in range(E):
            only = torch.full((E,), -4.0, device="cuda")
            only[e] = 0.0
            i, v = M.moe_route_topk(l, 1, score=score, bias=only, renormalize=False)
            assert bool((i == e).all())
            s[:, e] = v[:, 0].cpu().numpy()
        want = np.stack([np.lexsort((np.arange(E), -row))[:k] for row in s])
        assert np.array_equal(ids, want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group", [(64, 8), (256, 8), (93, 31), (510, 30)])
def test_groups_go_by_the_scores(score, E, n_group):
    # the one group with the largest sum of its two largest scores, in FP32, the lower group on equal sums
    l = close_logits(200, E, 0.4, seed=E)
    size = E // n_group
    for bias in (None, torch.zeros(E, device="cuda")):
        ids, _ = M.moe_route_topk(l, 2, score=score, bias=bias, n_group=n_group, topk_group=1, group_score="top2")
        every, w = [], []
        for lo in range(0, E, 32):                           # every expert's score, 32 at a time: the others' bias is lower
            up = torch.full((E,), -4.0, device="cuda")
            up[lo:lo + 32] = 0.0
            i, v = M.moe_route_topk(l, min(32, E - lo), score=score, bias=up, renormalize=False)
            every.append(i.cpu().numpy())
            w.append(v.cpu().numpy())
        s = np.empty((200, E), np.float32)
        np.put_along_axis(s, np.concatenate(every, 1).astype(np.int64), np.concatenate(w, 1), 1)
        top = -np.sort(-s.reshape(200, n_group, size), axis=2)[..., :2]
        sums = top[..., 0] + top[..., 1]                     # FP32
        assert np.array_equal(ids[:, 0].cpu().numpy() // size, sums.argmax(1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias_is_added_in_fp32(score):
    # o = s + b rounded once: the ids of every row are those of the FP32 sums of the returned scores
    E, k = 64, 64 // 2
    l = close_logits(300, E, 0.3, seed=7)
    bias = (torch.randint(-3, 4, (E,), generator=torch.Generator().manual_seed(1)).float() * 2.0 ** -22).cuda()
    s = np.empty((300, E), np.float32)
    for lo in (0, 32):
        up = torch.full((E,), -4.0, device="cuda")
        up[lo:lo + 32] = 0.0
        i, v = M.moe_route_topk(l, 32, score=score, bias=up, renormalize=False)
        np.put_along_axis(s, i.cpu().numpy().astype(np.int64), v.cpu().numpy(), 1)
    o = s + bias.cpu().numpy()[None, :]
    assert o.dtype == np.float32
    ids, _ = M.moe_route_topk(l, k, score=score, bias=bias)
    want = np.stack([np.lexsort((np.arange(E), -row))[:k] for row in o])
    assert np.array_equal(ids.cpu().numpy(), want)
