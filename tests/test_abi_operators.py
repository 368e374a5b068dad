"""Refusals and host-side answers of the routing of given logits and of the dense 4-bit products:
every call here is rejected or answered on the host, nothing is launched."""

import ctypes

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B

OK, ARG, SHAPE, WS = 0, 1, 2, 3
P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


def params(score=0, k=4, n_group=1, topk_group=1, group_score=0, renormalize=1, scale=1.0):
    return M.moe_route_params(score, k, n_group, topk_group, group_score, renormalize, scale)


def test_route_refusals(lib):
    def call(T=8, E=64, ld=64, type=0, x=P, b=None, ids=P, w=P, p=None, **kw):
        return lib.moe_route_topk(x, type, T, E, ld, params(**kw) if p is None else p, b, ids, w, None)
    assert call(T=0) == OK                                            # nothing to do, nothing launched
    assert call(T=0, x=None, ids=None, w=None) == OK
    for kw in (dict(T=-1), dict(T=1 << 31), dict(E=0, ld=0), dict(E=1025, ld=1025), dict(ld=63), dict(type=3),
               dict(type=-1), dict(ld=1 << 60),
               dict(k=0), dict(k=33), dict(E=8, k=9), dict(score=2), dict(renormalize=2), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(n_group=0), dict(n_group=3), dict(E=66, ld=66, n_group=33),
               dict(n_group=8, topk_group=0), dict(n_group=8, topk_group=9), dict(n_group=8, topk_group=1, k=9),
               dict(n_group=8, topk_group=1, group_score=2)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(x=ODD), dict(type=1, x=ODD), dict(ids=ODD), dict(w=ODD),
               dict(b=ODD)):
        assert call(**kw) == ARG, kw
    assert lib.moe_route_topk(P, 0, 8, 64, 64, None, None, P, P, None) == ARG


def test_route_backward_refusals(lib):
    def call(T=8, E=64, ld=64, ldo=64, type=0, x=P, ids=P, dw=P, out=P, **kw):
        return lib.moe_route_topk_backward(x, type, T, E, ld, params(**kw), ids, dw, out, ldo, None)
    assert call(T=0, x=None) == OK
    # groups and bias have no part in it
    assert call(T=0, n_group=0, topk_group=-5, group_score=9) == OK
    for kw in (dict(T=-1), dict(E=1025, ld=1025, ldo=1025), dict(ld=63), dict(ldo=63), dict(type=5), dict(k=0),
               dict(k=33), dict(E=4, k=5), dict(score=-1), dict(scale=float("inf"))):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(ids=None), dict(dw=None), dict(out=None), dict(x=ODD), dict(out=ODD), dict(dw=ODD)):
        assert call(**kw) == ARG, kw


def test_mxfp4_rows(lib):
    assert M.mxfp4_sf_bytes(1, 32) == 512 and M.mxfp4_sf_bytes(129, 160) == 2 * 2 * 512
    assert M.mxfp4_sf_bytes(0, 64) == 0 and M.mxfp4_sf_bytes(4, 48) == 0 and M.mxfp4_sf_bytes(-1, 64) == 0
    def q(x=P, type=1, rows=4, cols=64, ld=64, codes=P, sf=P):
        return lib.mxfp4_quantize_rows(x, type, rows, cols, ld, codes, sf, None)
    assert q(rows=0, x=None, codes=None, sf=None) == OK
    for kw in (dict(rows=-1), dict(cols=48, ld=48), dict(cols=0), dict(ld=32), dict(type=3), dict(cols=(1 << 20) + 32, ld=1 << 21)):
        assert q(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(codes=None), dict(sf=None), dict(x=ODD), dict(codes=ctypes.c_void_p(4104)),
               dict(sf=ctypes.c_void_p(4104))):
        assert q(**kw) == ARG, kw
    def d(codes=P, sf=P, rows=4, cols=64, out=P, type=1, ld=64):
        return lib.mxfp4_dequantize_rows(codes, sf, rows, cols, out, type, ld, None)
    assert d(rows=0, codes=None) == OK
    for kw in (dict(type=2), dict(ld=63), dict(cols=40, ld=64)):
        assert d(**kw) == SHAPE, kw
    for kw in (dict(codes=None), dict(sf=None), dict(out=None), dict(out=ODD)):
        assert d(**kw) == ARG, kw


@pytest.mark.parametrize("mx", [True, False])
def test_linear_refusals(lib, mx):
    def call(T=17, K=128, N=100, ldx=128, ldo=100, x=P, x_type=1, bias=None, out=P, out_type=1, ws=P, nbytes=1 << 20,
             codes=4096, sf=4096, g=4096):
        w = M.fp4_linear_weights(codes, sf, None if mx else g, N, K)
        if mx:
            return lib.mxfp4_linear(w, x, x_type, T, ldx, bias, out, out_type, ldo, ws, nbytes, None)
        return lib.nvfp4_linear(w, x, T, ldx, bias, out, out_type, ldo, ws, nbytes, None)
    assert call(T=0) == OK and call(T=0, x=None, out=None, ws=None, nbytes=0) == OK
    for kw in (dict(T=-1), dict(T=1 << 31), dict(N=0), dict(ldx=120), dict(ldo=99), dict(out_type=3), dict(K=80, ldx=80)):
        assert call(**kw) == SHAPE, kw
    if mx:
        assert call(x_type=4) == SHAPE
    else:
        assert call(K=96, ldx=96) == SHAPE and call(K=8256, ldx=8256) == SHAPE and call(ldx=132) == SHAPE
        assert call(g=None) == ARG and call(x=ctypes.c_void_p(4104)) == ARG
    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(x=ODD), dict(out=ODD), dict(bias=ODD),
               dict(ws=ctypes.c_void_p(4112)), dict(codes=None), dict(sf=None), dict(codes=4104), dict(sf=4104)):
        assert call(**kw) == ARG, kw
    size = lib.mxfp4_linear_workspace_bytes if mx else lib.nvfp4_linear_workspace_bytes
    need = size(17, 128)
    assert need >= 128 * 64 + (512 if mx else 1024) and need % 256 == 0
    assert call(nbytes=need - 1) == WS
    # few tokens need none
    assert size(1, 8192) == 0 and size(16, 2048) == 0 and size(16, 4096) > 0
    assert call(T=4, ws=ctypes.c_void_p(4112)) == ARG
    assert lib.mxfp4_linear_workspace_bytes(4, 48) == 0 and lib.nvfp4_linear_workspace_bytes(4, 96) == 0
    f = lib.mxfp4_linear if mx else lib.nvfp4_linear
    args = (P, 1, 17, 128) if mx else (P, 17, 128)
    assert f(None, *args, None, P, 1, 100, P, 1 << 20, None) == ARG


def test_python_checks():
    cpu = torch.zeros((4, 64))
    for call in (lambda: M.moe_route_topk(cpu, 2), lambda: M.moe_route_topk(cpu.double(), 2),
                 lambda: M.moe_route_topk(cpu[0], 2),
                 lambda: M.moe_route_topk_backward(cpu, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))),
                 lambda: M.mxfp4_quantize_rows(cpu), lambda: M.mxfp4_quantize_rows(cpu.int()),
                 lambda: M.mxfp4_dequantize_rows(torch.zeros((128, 32), dtype=torch.uint8),
                                                 torch.zeros(512, dtype=torch.uint8), 4, 64),
                 lambda: M.mxfp4_dequantize_rows(cpu, cpu, 4, 64, dtype=torch.float16),
                 lambda: M.mxfp4_weight_from_codes(torch.zeros((4, 32), dtype=torch.uint8),
                                                   torch.zeros((4, 3), dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()


def test_routing_parameters_are_those_of_the_call():
    scale = torch.tensor(2.5)
    p = M._route_params("sigmoid", 8, 4, 2, "top2", True, scale)
    assert (p.score, p.k, p.n_group, p.topk_group, p.group_score, p.renormalize, p.scale) == (1, 8, 4, 2, 1, 1, 2.5)
    scale += 1.0                                             # a parameter is its value, not its object
    assert M._route_params("sigmoid", 8, 4, 2, "top2", True, scale).scale == 3.5 and p.scale == 2.5
    assert M._route_params("softmax", 8, 1, 1, "max", 0, 1).renormalize == 0
    with pytest.raises(ValueError):
        M._route_params("relu", 8, 1, 1, "max", True, 1.0)
    with pytest.raises(ValueError):
        M._route_params("softmax", 8, 1, 1, "mean", True, 1.0)
    with pytest.raises(TypeError):
        M._route_params("softmax", 2.5, 1, 1, "max", True, 1.0)
