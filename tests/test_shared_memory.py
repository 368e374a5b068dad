"""Outputs in the memory of the input they are computed from.

The routing's gradient writes a row's zeros before it reads the logits, so it cannot be taken in place.  The product of few tokens reads x and writes its outputs in one kernel, so through the C ABI their rows have to lie
apart; the Python calls take a copy of x where they do not."""

import ctypes

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B

OK, ARG = 0, 1


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


@pytest.mark.parametrize("mx", [True, False])
def test_few_tokens_refuse_rows_they_read(lib, mx):
    def call(x, out, T=4, K=128, N=128, ldx=128, ldo=128, out_type=1):
        w = M.fp4_linear_weights(4096, 4096, None if mx else 4096, N, K)
        x, out = ctypes.c_void_p(x), ctypes.c_void_p(out)
        if mx:
            return lib.mxfp4_linear(w, x, 1, T, ldx, None, out, out_type, ldo, None, 0, None)
        return lib.nvfp4_linear(w, x, T, ldx, None, out, out_type, ldo, None, 0, None)
    base = 1 << 20
    assert call(base, base) == ARG                                   # in place
    assert call(base, base, T=1) == ARG
    assert call(base, base + 3 * 256 + 254) == ARG                   # the last element of x
    assert call(base, base - 4 * 256 + 2) == ARG                     # the first
    assert call(base, base + 254, ldx=512, ldo=512) == ARG           # column blocks that meet
    assert call(base + 256, base + 2, ldx=512, ldo=512) == ARG
    assert call(base, base + 768 + 2, ldx=512, ldo=512) == ARG       # out's rows end in x's next ones
    assert call(base, base + 512, ldx=512, ldo=256) == ARG           # rows of two pitches: out's second is x's second
    assert call(base, base + 256, T=3, ldx=512, ldo=384, out_type=0) == ARG


def test_share_memory():
    buf = torch.empty(4096, dtype=torch.bfloat16)
    rows = lambda at, ld, T=4, n=128: torch.as_strided(buf, (T, n), (ld, 1), at)   # noqa: E731
    share = M._share_memory
    assert share(rows(0, 128), rows(0, 128)) and share(rows(0, 128), rows(511, 128))
    assert not share(rows(0, 128), rows(512, 128)) and not share(rows(512, 128), rows(0, 128))
    assert not share(rows(0, 256), rows(128, 256)) and not share(rows(128, 256), rows(0, 256))
    assert share(rows(0, 256), rows(127, 256)) and share(rows(0, 256), rows(129, 256))
    assert not share(rows(0, 256), rows(640, 256)) and share(rows(0, 256), rows(641, 256))
    assert share(rows(0, 200, T=1), rows(127, 300, T=1)) and not share(rows(0, 200, T=1), rows(128, 300, T=1))
    assert not share(rows(0, 128, T=0), rows(0, 128, T=0))


def test_routing_gradient_refuses_its_logits_memory(lib):
    p = M.moe_route_params(0, 4, 1, 1, 0, 1, 1.0)
    base = 1 << 20

    def call(x, out, T=8, E=64, ld=64, ldo=64):
        x, out = ctypes.c_void_p(x), ctypes.c_void_p(out)
        return lib.moe_route_topk_backward(x, 0, T, E, ld, p, ctypes.c_void_p(4096), ctypes.c_void_p(4096), out, ldo, None)
    for score in (0, 1):
        for renormalize in (0, 1):
            p.score, p.renormalize = score, renormalize
            assert call(base, base) == ARG and call(base, base, T=1) == ARG
            assert call(base, base + 252, ld=128, ldo=128) == ARG and call(base, base + 8 * 256 - 4) == ARG
            assert call(base, base + 4096, T=64, ld=64, ldo=128) == ARG


@pytest.mark.gpu
def test_routing_gradient_beside_its_logits(lib):
    # logits and gradient as column blocks of one buffer
    both = torch.zeros(300, 256, device="cuda")
    l = torch.randn(300, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    both[:, :128] = l
    dw = torch.randn(300, 8, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    for score in (0, 1):
        for renormalize in (0, 1):
            name = "sigmoid" if score else "softmax"
            ids, _ = M.moe_route_topk(l, 8, score=name, renormalize=bool(renormalize))
            want = M.moe_route_topk_backward(l, ids, dw, score=name, renormalize=bool(renormalize))
            p = M.moe_route_params(score, 8, 1, 1, 0, renormalize, 1.0)
            status = lib.moe_route_topk_backward(both.data_ptr(), 0, 300, 128, 256, p, ids.data_ptr(), dw.data_ptr(),
                                                 both[:, 128:].data_ptr(), 256, torch.cuda.current_stream().cuda_stream)
            assert status == OK and torch.equal(both[:, 128:], want) and torch.equal(both[:, :128], l)


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T", [1, 5, 16, 40, 2400])
def test_product_in_place(lib, mx, T):
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, 2048, device="cuda", generator=g).to(torch.bfloat16)
    w = (0.05 * torch.randn(2048, 2048, device="cuda", generator=g)).to(torch.bfloat16)
    linear, wq = (M.mxfp4_linear, M.mxfp4_quantize_weight(w)) if mx else (M.nvfp4_linear, M.nvfp4_quantize_weight(w))
    want = linear(x, wq)
    same = x.clone()
    assert linear(same, wq, out=same) is same and torch.equal(same, want)
    s = torch.cuda.Stream()
    again = x.clone()
    s.wait_stream(torch.cuda.current_stream())
    linear(again, wq, out=again, stream=s)
    s.synchronize()
    assert torch.equal(again, want)
    # column blocks of one buffer lie apart; blocks that meet do not
    for at in (2048, 1024):
        both = torch.zeros(T, 4096, dtype=torch.bfloat16, device="cuda")
        both[:, :2048] = x
        linear(both[:, :2048], wq, out=both[:, at:at + 2048])
        assert torch.equal(both[:, at:at + 2048], want)
        if at == 2048:
            assert torch.equal(both[:, :2048], x)
    assert M.nvfp4_get_device_error() == 0
