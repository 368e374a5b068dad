"""Refusals of the balance loss and its gradient: every call here is rejected on the host, nothing is launched."""

import ctypes

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from test_devices import Tensor, device_0  # noqa: F401

OK, ARG, SHAPE = 0, 1, 2
V = ctypes.c_void_p
P, ODD = V(4096), V(4097)
FAR = V(1 << 30)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


SHAPES = (dict(T=-1), dict(T=1 << 31), dict(E=0, ld=0), dict(E=1025, ld=1025), dict(ld=63), dict(ld=1 << 60), dict(type=3),
          dict(type=-1), dict(score=2), dict(score=-1), dict(k=0), dict(k=33), dict(E=4, k=5), dict(S=0), dict(S=1 << 27, off=P),
          dict(S=2))


def test_refusals(lib):
    def call(T=8, E=64, ld=64, type=0, score=0, x=P, ids=P, k=4, mask=None, off=None, S=1, loss=P, counts=P, probs=P, tokens=P,
             ws=P, n=1 << 24):
        return lib.moe_balance_loss(x, type, T, E, ld, score, ids, k, mask, off, S, loss, counts, probs, tokens, ws, n, None)
    for kw in SHAPES:
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(ids=None), dict(loss=None), dict(counts=None), dict(probs=None), dict(tokens=None),
               dict(x=ODD), dict(type=1, x=ODD), dict(ids=ODD), dict(off=ODD), dict(loss=ODD), dict(counts=ODD),
               dict(probs=ODD), dict(tokens=ODD), dict(T=0, loss=None), dict(ws=V(4112)),
               dict(T=5000, ws=None)):
        assert call(**kw) == ARG, kw
    size = lib.moe_balance_workspace_bytes
    assert size(1024, 64, 32) == 0 and size(8, 1024, 1) == 0                  # few tokens need none
    need = size(5000, 64, 3)
    assert need > 0 and need % 256 == 0 and call(T=5000, S=3, off=P, n=need - 1) == 3
    assert size(8, 64, 33) > 0 and size(-1, 64, 1) == 0 and size(8, 0, 1) == 0 and size(8, 1025, 1) == 0 and size(8, 64, 0) == 0


def test_backward_refusals(lib):
    def call(T=8, E=64, ld=64, ldo=64, type=0, score=0, x=P, k=4, mask=None, off=None, S=1, counts=P, tokens=P, dloss=P,
             out=FAR, add=0):
        return lib.moe_balance_loss_backward(x, type, T, E, ld, score, k, mask, off, S, counts, tokens, dloss, out, ldo, add, None)
    assert call(T=0) == OK and call(T=0, x=None, counts=None, out=None) == OK
    for kw in SHAPES + (dict(ldo=63), dict(add=2), dict(add=-1), dict(ldo=1 << 60)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(counts=None), dict(tokens=None), dict(dloss=None), dict(out=None), dict(x=ODD), dict(out=ODD),
               dict(counts=ODD), dict(tokens=ODD), dict(dloss=ODD), dict(off=ODD), dict(out=P), dict(add=1, out=P),
               dict(out=V(4096 + 8 * 64 * 4 - 4))):
        assert call(**kw) == ARG, kw


f32, i32 = torch.float32, torch.int32


def logits(T=8, E=64, dtype=f32):
    t = Tensor(dtype, T, E)
    t.get_device = lambda: 0
    return t


@pytest.mark.parametrize("make", [
    lambda: M.moe_balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32)),
    lambda: M.moe_balance_loss(logits(dtype=torch.float64), Tensor(i32, 8, 2)),
    lambda: M.moe_balance_loss(logits(), Tensor(torch.int64, 8, 2)),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 7, 2)),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 8)),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 8, 2), score="relu"),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 8, 2), mask=Tensor(f32, 8)),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 8, 2), mask=Tensor(torch.bool, 7)),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 8, 2), seq_offsets=Tensor(i32, 1)),
    lambda: M.moe_balance_loss(logits(), Tensor(i32, 8, 2), seq_offsets=Tensor(torch.int64, 3)),
    lambda: M.moe_balance_loss(Tensor(f32, 8, 64), Tensor(i32, 8, 2)),
    lambda: M.moe_balance_loss_backward(logits(), 2, Tensor(i32, 1, 63), Tensor(i32, 1), Tensor(f32, 1)),
    lambda: M.moe_balance_loss_backward(logits(), 2, Tensor(i32, 1, 64), Tensor(i32, 2), Tensor(f32, 1)),
    lambda: M.moe_balance_loss_backward(logits(), 2, Tensor(i32, 1, 64), Tensor(i32, 1), Tensor(torch.float64, 1)),
    lambda: M.moe_balance_loss_backward(logits(), 2, Tensor(i32, 1, 64), Tensor(i32, 1), Tensor(f32, 1),
                                        dlogits=logits(dtype=torch.bfloat16)),
    lambda: M.moe_balance_loss_backward(logits(), 2, Tensor(i32, 1, 64), Tensor(i32, 1), Tensor(f32, 1), dlogits=logits(E=65)),
    lambda: M.moe_balance_loss_backward(logits(), (1 << 32) + 2, Tensor(i32, 1, 64), Tensor(i32, 1), Tensor(f32, 1),
                                        dlogits=logits()),
    lambda: M.moe_balance_loss_backward(Tensor(f32, 8, 64), 2, Tensor(i32, 1, 64), Tensor(i32, 1), Tensor(f32, 1)),
])
def test_python_refusals(make, device_0):  # noqa: F811
    with pytest.raises(ValueError):
        make()
