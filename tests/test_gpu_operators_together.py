"""The routing calls and the dense products as a program uses them: in a captured graph, from several streams and
threads at once, with the weights of a checkpoint."""

import threading

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import mxfp4 as X
from oracle import quant as Q
from _helpers import GEMM_REL_L2

pytestmark = pytest.mark.gpu
ROUTES = [dict(), dict(score="sigmoid", renormalize=False), dict(renormalize=False, scale=2.0),
          dict(score="sigmoid", n_group=8, topk_group=4, group_score="top2", scale=2.5)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def make(T, E, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(T, E, device="cuda", generator=g), 0.05 * torch.randn(E, device="cuda", generator=g)


def gradient_kw(kw):
    return {n: kw[n] for n in ("score", "renormalize", "scale") if n in kw}


@pytest.mark.parametrize("kw", ROUTES)
@pytest.mark.parametrize("T", [1, 300])
def test_routing_in_a_captured_graph(kw, T):
    l, bias = make(T, 128, 1)
    dw = torch.randn(T, 6, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    M.moe_route_topk(l, 6, bias=bias, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, w = M.moe_route_topk(l, 6, bias=bias, **kw)
        dl = M.moe_route_topk_backward(l, ids, dw, **gradient_kw(kw))
    for seed in (3, 4):                                      # the graph reads the inputs of each replay
        fresh, fresh_bias = make(T, 128, seed)
        l.copy_(fresh)
        bias.copy_(fresh_bias)
        for t in (ids, w, dl):
            t.zero_()
        g.replay()
        want = M.moe_route_topk(l, 6, bias=bias, **kw)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
        assert torch.equal(dl, M.moe_route_topk_backward(l, ids, dw, **gradient_kw(kw)))
    assert M.nvfp4_get_device_error() == 0


def work(seed):
    """One of everything, of a size of its own."""
    T = 50 + 700 * (seed % 3)
    l, bias = make(T, 256, seed)
    kw = ROUTES[seed % len(ROUTES)]
    ids, w = M.moe_route_topk(l, 8, bias=bias, **kw)
    dl = M.moe_route_topk_backward(l, ids, w, **gradient_kw(kw))
    x = l.to(torch.bfloat16)
    wt = x[:48].repeat(3, 1).contiguous()
    mx, nv = M.mxfp4_quantize_weight(wt), M.nvfp4_quantize_weight(wt)
    one = x[:1].contiguous()
    return [ids, w, dl, *M.mxfp4_quantize_rows(x), M.mxfp4_linear(x, mx), M.nvfp4_linear(x, nv), M.mxfp4_linear(one, mx),
            M.nvfp4_linear(one, nv)]


def test_several_streams_and_threads_at_once():
    count, turns = 4, 6
    want = [work(seed) for seed in range(count)]
    torch.cuda.synchronize()
    bad = []

    def run(seed):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(turns):
                got = work(seed)
                torch.cuda.current_stream().synchronize()
                bad.extend(seed for a, b in zip(got, want[seed]) if not torch.equal(a, b))

    threads = [threading.Thread(target=run, args=(seed,)) for seed in range(count)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    # and interleaved by one thread over two streams
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(turns):
        for seed, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((seed, work(seed)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for seed, tensors in got for a, b in zip(tensors, want[seed]))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T,N,K", [(1, 70, 416), (16, 300, 2048), (40, 129, 96), (2400, 2100, 288)])
def test_products_with_a_checkpoints_codes(T, N, K):
    # weights that are MXFP4 already, every code and a range of scales; the tolerance of the products' tests
    rng = np.random.default_rng(N)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    scales = rng.integers(118, 133, (N, K // 32), dtype=np.uint8)
    w = M.mxfp4_weight_from_codes(torch.from_numpy(Q.pack_nibbles(codes)).cuda(), torch.from_numpy(scales).cuda())
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    y = M.mxfp4_linear(x, w, out_dtype=torch.float32).double().cpu().numpy()
    a = X.dequantize_rows(*X.quantize_rows(x.float().cpu().numpy()))
    b = X.dequantize_rows(codes, scales)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    err = np.abs(y - want)
    assert np.all(err <= 2.0 ** -20 * size + 2.0 ** -24 * np.abs(want))
    assert np.linalg.norm(err) <= GEMM_REL_L2 * np.linalg.norm(want)
