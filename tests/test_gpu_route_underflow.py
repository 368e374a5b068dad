"""Sigmoid scores of very low logits.

Renormalised weights are ratios of scores and do not go to zero with them; neither do their gradients.  Tolerances: those
of tests/test_gpu_route_topk.py (5e-6 of a weight, 2e-5 of a gradient's terms; FP32's smallest values beside them).
Scores by themselves are FP32 values: below 2^-126 they keep what its subnormals hold, half a unit of 2^-149, and
the two units that the exponential may be off."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import route_topk as R

pytestmark = pytest.mark.gpu
W_REL, G_REL = 5e-6, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def rows(E, seed):
    """Logits around -95 (and beside that range), spread 3; some rows reach into it from ordinary values."""
    g = torch.Generator().manual_seed(seed)
    l = 3.0 * torch.randn(48, E, generator=g)
    l += torch.tensor([-95.0, -88.0, -100.0, -104.0, -120.0, -300.0, -340.0, -80.0, -40.0, -17.0, 0.0, 30.0]).repeat(4)[:, None]
    l[36:, : E // 2] = l[36:, : E // 2] - 90.0
    l[5, 1] = -float("inf")
    return l.cuda()


def terms(l, ids, dw, scale):
    """Magnitudes that a renormalised gradient is the difference of."""
    i = ids.astype(np.int64)
    q = R.weights(l, ids, "sigmoid", True, 1.0)
    g = np.abs(dw * scale)
    out = np.zeros_like(l)
    np.put_along_axis(out, i, q * (g + (g * q).sum(1, keepdims=True)), 1)
    return out


@pytest.mark.parametrize("E,k", [(8, 8), (48, 6), (128, 9), (250, 20), (1024, 32)])
def test_renormalised(E, k):
    l = rows(E, E)
    ids, w = M.moe_route_topk(l, k, score="sigmoid", scale=2.5)
    l64, i, w = l.cpu().double().numpy(), ids.cpu().numpy(), w.cpu().double().numpy()
    want_ids, want = R.route(l64, k, score="sigmoid", scale=2.5)
    assert np.array_equal(i, want_ids)
    assert np.all(np.abs(w - want) <= W_REL * want + 1e-30)
    assert np.allclose(w.sum(1), 2.5, rtol=1e-5)
    dw = torch.randn(48, k, generator=torch.Generator().manual_seed(3)).cuda()
    got = M.moe_route_topk_backward(l, ids, dw, score="sigmoid", scale=2.5).cpu().double().numpy()
    d64 = dw.cpu().double().numpy()
    exact = R.backward(l64, i, d64, "sigmoid", True, 2.5)
    assert np.all(np.abs(got - exact) <= G_REL * terms(l64, i, d64, 2.5) + 2.0 ** -24 * np.abs(exact) + 1e-30)
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_renormalised_in_16_bits(dtype):
    l = rows(64, 2).to(dtype)
    ids, w = M.moe_route_topk(l, 8, score="sigmoid")
    want = R.weights(l.cpu().double().numpy(), ids.cpu().numpy(), "sigmoid", True, 1.0)
    assert np.all(np.abs(w.cpu().double().numpy() - want) <= W_REL * want + 1e-30)


def test_not_renormalised():
    l = rows(48, 1)
    ids, w = M.moe_route_topk(l, 6, score="sigmoid", renormalize=False)
    want = R.weights(l.cpu().double().numpy(), ids.cpu().numpy(), "sigmoid", False, 1.0)
    assert np.all(np.abs(w.cpu().double().numpy() - want) <= W_REL * want + 2.5 * 2.0 ** -149)


def test_weights_as_low_as_64_bits_hold():
    l = (3.0 * torch.randn(20, 40, generator=torch.Generator().manual_seed(4)) - 690.0).cuda()
    ids, w = M.moe_route_topk(l, 8, score="sigmoid")
    want = R.weights(l.cpu().double().numpy(), ids.cpu().numpy(), "sigmoid", True, 1.0)
    assert np.all(np.abs(w.cpu().double().numpy() - want) <= W_REL * want) and np.allclose(want.sum(1), 1.0)


def test_scores_in_units_of_the_last_place():
    # t = e^-|l| within 2^-22 (two units), 1 + t and its reciprocal y within 2^-24 each: y (l >= 0) is within 4 units of
    # 2^-24 of the sigmoid, t y (l < 0) within 9
    l = torch.linspace(-86.0, 30.0, 116 * 512, dtype=torch.float64).float().reshape(-1, 32).cuda()
    ids, w = M.moe_route_topk(l, 32, score="sigmoid", renormalize=False)
    l64 = np.take_along_axis(l.cpu().double().numpy(), ids.cpu().numpy().astype(np.int64), 1)
    want = 1.0 / (1.0 + np.exp(-l64))
    units = np.abs(w.cpu().double().numpy() - want) / want * 2.0 ** 24
    assert units[l64 >= 0].max() <= 4.0 and units[l64 < 0].max() <= 9.0


def test_nothing_left_of_the_sum():
    # masked, or as low as a mask by the type's lowest value is: no weights and no gradient
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        l = torch.full((3, 16), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        l[1] = -float("inf")
        l[2] = -710.0
        ids, w = M.moe_route_topk(l, 4, score="sigmoid")
        assert ids.tolist() == [[0, 1, 2, 3]] * 3 and not bool(w.any())
        assert not bool(M.moe_route_topk_backward(l, ids, torch.ones_like(w), score="sigmoid").any())
