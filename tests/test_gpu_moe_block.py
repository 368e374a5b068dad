"""The example block (examples/moe_block.py): its parts run together as a model has them."""

import os
import sys

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import route_topk as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    B.build()
    import moe_block
    return moe_block.MoEBlock(H=512, I=256, E=64, k=6, n_group=8, topk_group=4)


def make_x(T, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(T, 512, device="cuda", generator=g).to(torch.bfloat16)


def test_forward_is_its_parts(block):
    x = make_x(200)
    y = block.forward(x)
    _, logits, ids = block.saved
    l = logits.double().cpu().numpy()
    # the routing against the oracle, where no two of its values lie within rounding
    want, _ = R.route(l, 6, score="sigmoid", bias=block.bias.double().cpu().numpy(), n_group=8, topk_group=4,
                      group_score="top2")
    same = (ids.cpu().numpy() == want).all(1)
    assert same.mean() > 0.95
    w = torch.from_numpy(R.weights(l, ids.cpu().numpy(), "sigmoid", True, 2.5)).float().cuda()
    again = block.experts.forward(x, ids, w) + block.shared(x)
    # the weights differ by FP32 rounding: a BF16 product or sum may round the other way
    assert float((y.float() - again.float()).norm()) <= 2.0 ** -8 * float(again.float().norm())
    assert M.nvfp4_get_device_error() == 0


def test_batch_invariance(block):
    x = make_x(300)
    y = block.forward(x)
    for lo, hi in ((0, 1), (5, 21), (100, 300)):
        assert torch.equal(block.forward(x[lo:hi].contiguous()), y[lo:hi])


def test_backward_reaches_the_router(block):
    x = make_x(256, seed=2)
    y = block.forward(x, train=True)
    dout = torch.randn(*y.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    dx, dw1, dw2, dw_router = block.backward(dout)
    _, logits, ids = block.saved
    block.forward(x, train=True)
    _, _, _, dprob = block.experts.backward(dout)
    dl = R.backward(logits.double().cpu().numpy(), ids.cpu().numpy(), dprob.double().cpu().numpy(), "sigmoid", True, 2.5)
    want = dl.T @ x.double().cpu().numpy()
    got = dw_router.double().cpu().numpy()
    # FP32 logits' gradient (2e-5 of its terms) and an FP32 product over 256 tokens
    assert np.linalg.norm(got - want) <= 1e-4 * np.linalg.norm(want)
    assert dx.shape == x.shape and bool(torch.isfinite(dx.float()).all())


def test_balance_moves_the_bias(block):
    block.forward(make_x(400))
    before = block.bias.clone()
    load = block.balance(0.01)
    moved = block.bias - before
    assert bool((moved[load > load.mean()] < 0).all()) and bool((moved[load < load.mean()] > 0).all())
    block.bias.copy_(before)
