"""Refusals of the adapters' calls: every call here is rejected or answered on the host, nothing is launched."""

import ctypes

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from test_devices import Tensor, device_0  # noqa: F401

OK, ARG, SHAPE, WS = 0, 1, 2, 3
V = ctypes.c_void_p
X, Y, OUT, P, ODD = V(1 << 20), V(1 << 30), V(1 << 31), V(4096), V(4097)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


def adapters(down=4096, up=4096, scale=None, type=1, L=3, R=16, K=64, N=40):
    return M.lora_adapters(down, up, scale, type, L, R, K, N)


BAD_SHAPE = (dict(type=0), dict(type=3), dict(L=0), dict(L=1025), dict(R=0), dict(R=12), dict(R=136), dict(K=0), dict(K=60),
             dict(K=(1 << 20) + 8), dict(N=0), dict(N=(1 << 20) + 1))
BAD_POINTER = (dict(down=None), dict(up=None), dict(down=4104), dict(up=4104), dict(scale=4097))


def test_refusals(lib):
    def call(T=300, x=X, ldx=64, ids=P, y=Y, ldy=40, out=OUT, ldo=40, out_type=1, h=None, ws=P, n=1 << 20, **kw):
        return lib.lora_add(adapters(**kw), x, T, ldx, ids, y, ldy, out, ldo, out_type, h, ws, n, None)
    assert call(T=0) == OK and call(T=0, x=None, ids=None, y=None, out=None, ws=None, n=0) == OK
    for kw in BAD_SHAPE + (dict(T=-1), dict(T=1 << 31), dict(ldx=56), dict(ldx=68), dict(ldy=39), dict(ldo=39), dict(out_type=3),
                           dict(out_type=-1), dict(ldx=1 << 60), dict(ldo=1 << 60)):
        assert call(**kw) == SHAPE, kw
    for kw in BAD_POINTER + (dict(x=None), dict(ids=None), dict(y=None), dict(out=None), dict(ws=None), dict(x=V((1 << 20) + 8)),
                             dict(ids=ODD), dict(y=ODD), dict(out=ODD), dict(out_type=0, out=V((1 << 31) + 2)),
                             dict(h=V(4104)), dict(ws=V(4112)),
                             dict(out=V((1 << 30) + 2)), dict(out=Y, ldo=48), dict(out=V((1 << 30) + 299 * 80 + 78)),
                             dict(y=X, out=X), dict(out=X), dict(out=V((1 << 20) + 300 * 128 - 2))):
        assert call(**kw) == ARG, kw
    need = lib.lora_add_workspace_bytes(300, 3)
    assert need >= 4 * 300 and need % 256 == 0 and call(n=need - 1) == WS
    assert lib.lora_add(None, X, 4, 64, P, Y, 40, OUT, 40, 1, None, None, 0, None) == ARG
    # few tokens need no workspace; sizes that are refused need none
    assert lib.lora_add_workspace_bytes(256, 1024) == 0 and lib.lora_add_workspace_bytes(257, 1) > 0
    assert lib.lora_add_workspace_bytes(-1, 3) == 0 and lib.lora_add_workspace_bytes(300, 1025) == 0


def test_backward_refusals(lib):
    def call(T=300, dy=Y, lddy=40, x=X, ldx=64, h=P, ids=P, dx=OUT, lddx=64, dx_type=1, add=0, ddown=P, dup=P, ws=P, n=1 << 26, **kw):
        return lib.lora_add_backward(adapters(**kw), dy, lddy, x, ldx, h, ids, T, dx, lddx, dx_type, add, ddown, dup, ws, n, None)
    for kw in BAD_SHAPE + (dict(type=2), dict(T=-1), dict(T=1 << 31), dict(lddy=39), dict(ldx=56), dict(ldx=68), dict(lddx=63),
                           dict(dx_type=3), dict(add=2), dict(lddx=1 << 60)):
        assert call(**kw) == SHAPE, kw
    for kw in BAD_POINTER + (dict(dy=None), dict(x=None), dict(h=None), dict(ids=None), dict(dx=None), dict(ddown=None),
                             dict(dup=None), dict(ws=None), dict(dy=ODD), dict(x=V((1 << 20) + 8)), dict(h=V(4104)), dict(ids=ODD),
                             dict(dx=ODD), dict(ddown=ODD), dict(dup=ODD), dict(ws=V(4112)), dict(dx=X), dict(dx=Y),
                             dict(dx=V((1 << 30) + 300 * 80 - 2)), dict(add=1, dx=X)):
        assert call(**kw) == ARG, kw
    need = lib.lora_add_backward_workspace_bytes(300, 3, 16, 64, 40)
    assert need >= 300 * (4 + 64) and need % 256 == 0 and call(n=need - 1) == WS
    size = lib.lora_add_backward_workspace_bytes
    assert size(0, 3, 16, 64, 40) == 0 and size(9, 3, 12, 64, 40) == 0 and size(9, 3, 16, 60, 40) == 0 and size(9, 3, 16, 64, 0) == 0
    assert lib.lora_add_backward(None, Y, 40, X, 64, P, P, 4, OUT, 64, 1, 0, P, P, P, 1 << 20, None) == ARG


f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


def here(t):
    """A tensor of the binding's current device, cuda:0."""
    t.get_device = lambda: 0
    return t


def set_of(dtype=bf16, L=3, R=16, K=64, N=40, up=None, scale=None):
    return M.LoRAAdapters(Tensor(dtype, L, R, K), up or Tensor(dtype, L, N, R), scale or Tensor(f32, L))


x, y, ids, h = (lambda: here(Tensor(bf16, 9, 64))), (lambda: here(Tensor(bf16, 9, 40))), Tensor(i32, 9), Tensor(f32, 9, 16)


@pytest.mark.parametrize("make", [
    lambda: M.LoRAAdapters(torch.zeros(3, 16, 64, dtype=bf16), torch.zeros(3, 40, 16, dtype=bf16)),
    lambda: set_of(f32),
    lambda: set_of(up=Tensor(bf16, 3, 40, 8)),
    lambda: set_of(up=Tensor(torch.float16, 3, 40, 16)),
    lambda: set_of(up=Tensor(bf16, 40, 16)),
    lambda: set_of(scale=Tensor(bf16, 3)),
    lambda: set_of(scale=Tensor(f32, 4)),
    lambda: M.lora_add(y(), here(Tensor(torch.float16, 9, 64)), set_of(), ids),
    lambda: M.lora_add(y(), here(Tensor(bf16, 9, 72)), set_of(), ids),
    lambda: M.lora_add(here(Tensor(bf16, 9, 41)), x(), set_of(), ids),
    lambda: M.lora_add(here(Tensor(bf16, 8, 40)), x(), set_of(), ids),
    lambda: M.lora_add(here(Tensor(torch.float64, 9, 40)), x(), set_of(), ids),
    lambda: M.lora_add(y(), x(), set_of(), Tensor(torch.int64, 9)),
    lambda: M.lora_add(y(), x(), set_of(), Tensor(i32, 8)),
    lambda: M.lora_add(y(), x(), set_of(), ids, out=here(Tensor(f32, 9, 40))),
    lambda: M.lora_add(y(), x(), set_of(), ids, out=here(Tensor(bf16, 9, 48))),
    lambda: M.lora_add(y(), Tensor(bf16, 9, 64), set_of(), ids),
    lambda: M.lora_add(Tensor(bf16, 9, 40), x(), set_of(), ids),
    lambda: M.lora_add_backward(y(), x(), h, set_of(torch.float16), ids),
    lambda: M.lora_add_backward(here(Tensor(f32, 9, 40)), x(), h, set_of(), ids),
    lambda: M.lora_add_backward(y(), x(), Tensor(f32, 9, 8), set_of(), ids),
    lambda: M.lora_add_backward(y(), x(), Tensor(bf16, 9, 16), set_of(), ids),
    lambda: M.lora_add_backward(y(), x(), h, set_of(), ids, dx=here(Tensor(bf16, 9, 40))),
    lambda: M.lora_add_backward(Tensor(bf16, 9, 40), x(), h, set_of(), ids),
])
def test_python_refusals(make, device_0):  # noqa: F811
    with pytest.raises(ValueError):
        make()
