"""The balance loss and the adapters as a program uses them: around a MoE block, in a captured graph, from several streams
and threads at once."""

import threading

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import balance as OB
from oracle import lora as OL
from oracle import quant as Q

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def values(t):
    return t.detach().cpu().double().numpy()


def batch(T, E, k, K, N, R, L, seed, ordered=False):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    d = dict(logits=n(T, E), x=n(T, K).to(BF16), y=n(T, N).to(BF16), dy=n(T, N).to(BF16), dloss=n(3),
             ids=n(T, E).topk(k).indices.to(torch.int32), down=(n(L, R, K) / K ** 0.5).to(BF16), up=(0.1 * n(L, N, R)).to(BF16),
             scale=n(L).abs(), mask=n(T) > -1.0, who=torch.randint(-1, L, (T,), device="cuda", generator=g).to(torch.int32))
    if ordered:
        d["who"] = d["who"].sort().values
    cut = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device="cuda")
    return d, cut


def everything(d, cut, k, adapters):
    b = M.moe_balance_loss(d["logits"], d["ids"], score="sigmoid", mask=d["mask"], seq_offsets=cut)
    dl = M.moe_balance_loss_backward(d["logits"], k, b.counts, b.tokens, d["dloss"], score="sigmoid", mask=d["mask"], seq_offsets=cut)
    out, h = M.lora_add(d["y"], d["x"], adapters, d["who"], save_for_backward=True)
    return [*b, dl, out, h, M.lora_add(d["y"], d["x"], adapters, d["who"]), *M.lora_add_backward(d["dy"], d["x"], h, adapters, d["who"])]


SIZES = [(9, 64, 4, 256, 130, 16, 3), (300, 128, 8, 520, 96, 24, 5), (3000, 64, 6, 1032, 264, 16, 4), (2500, 40, 4, 256, 203, 64, 3), (9000, 130, 6, 128, 72, 128, 4)]


@pytest.mark.parametrize("size", SIZES)
def test_in_a_captured_graph(size):
    k = size[2]
    d, cut = batch(*size, seed=1)
    adapters = M.LoRAAdapters(d["down"], d["up"], d["scale"])
    everything(d, cut, k, adapters)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = everything(d, cut, k, adapters)
    for seed in (2, 3):                                     # the graph reads the inputs of each replay, and the adapters' tensors
        fresh, _ = batch(*size, seed=seed, ordered=seed == 3)
        for name in d:
            d[name].copy_(fresh[name])
        for t in got:
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, everything(d, cut, k, adapters)))
    assert M.nvfp4_get_device_error() == 0


def test_two_graphs_of_one_pool():
    graphs, outs, kept = [], [], []
    pool = torch.cuda.graph_pool_handle()
    for i, size in enumerate(SIZES[1:3]):
        d, cut = batch(*size, seed=i)
        adapters = M.LoRAAdapters(d["down"], d["up"], d["scale"])
        everything(d, cut, size[2], adapters)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append([t.clone() for t in everything(d, cut, size[2], adapters)])
        graphs.append(g)
        kept.append((d, cut, size[2], adapters))
    for turn in (0, 1, 1, 0):
        graphs[turn].replay()
        got = [t.clone() for t in outs[turn]]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, everything(*kept[turn])))


def test_several_streams_and_threads_at_once():
    cases = []
    for i, size in enumerate(SIZES):
        d, cut = batch(*size, seed=10 + i)
        adapters = M.LoRAAdapters(d["down"], d["up"], d["scale"])
        cases.append((d, cut, size[2], adapters))
    want = [everything(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got = everything(*cases[i])
                torch.cuda.current_stream().synchronize()
                bad.extend(i for a, b in zip(got, want[i]) if not torch.equal(a, b))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    # a stream given to the call, its buffers allocated for it
    s = torch.cuda.Stream()
    d, cut, k, adapters = cases[2]
    s.wait_stream(torch.cuda.current_stream())
    out, h = M.lora_add(d["y"], d["x"], adapters, d["who"], save_for_backward=True, stream=s)
    grads = M.lora_add_backward(d["dy"], d["x"], h, adapters, d["who"], stream=s)
    b = M.moe_balance_loss(d["logits"], d["ids"], score="sigmoid", mask=d["mask"], seq_offsets=cut, stream=s)
    dl = M.moe_balance_loss_backward(d["logits"], k, b.counts, b.tokens, d["dloss"], score="sigmoid", mask=d["mask"], seq_offsets=cut, stream=s)
    s.synchronize()
    assert all(torch.equal(a, w) for a, w in zip([*b, dl, out, h], want[2])) and all(torch.equal(a, w) for a, w in zip(grads, want[2][8:]))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T", [6, 400, 4000])
@pytest.mark.parametrize("who", ["alternating", "in a row", "backwards", "one and none"])
def test_any_order_of_requests(T, who):
    d, _ = batch(T, 8, 2, 520, 104, 32, 6, seed=T)
    ids = {"alternating": torch.arange(T) % 6, "in a row": torch.arange(T) * 6 // T, "backwards": 5 - torch.arange(T) * 6 // T,
           "one and none": torch.where(torch.arange(T) % 97 == 5, -1, 4)}[who].to(torch.int32).cuda()
    adapters = M.LoRAAdapters(d["down"], d["up"], d["scale"])
    got, h = M.lora_add(d["y"], d["x"], adapters, ids, save_for_backward=True)
    # the same rows one adapter at a time, alone: the same bits
    for a in range(-1, 6):
        rows = (ids == a).nonzero().flatten()
        if rows.numel():
            one, one_h = M.lora_add(d["y"][rows], d["x"][rows], adapters, ids[rows], save_for_backward=True)
            assert torch.equal(got[rows], one) and torch.equal(h[rows], one_h)
    dx, ddown, dup = M.lora_add_backward(d["dy"], d["x"], h, adapters, ids)
    want = OL.backward(values(d["dy"]), values(d["x"]), values(h), values(d["down"]), values(d["up"]), values(d["scale"]), ids.cpu().numpy())
    for g, w, most in ((dx, want[0], 2.0 ** -8), (ddown, want[1], 2.0 ** -17), (dup, want[2], 2.0 ** -17)):
        assert np.linalg.norm(values(g) - w) <= most * np.linalg.norm(w)


def test_rows_without_an_adapter_keep_their_bits():
    for T in (5, 600, 4000):
        y = torch.zeros(T, 72, device="cuda").neg().to(BF16)      # -0
        y[:, 3] = float("nan")
        x, ids = torch.randn(T, 64, device="cuda").to(BF16), torch.full((T,), -1, dtype=torch.int32, device="cuda")
        ids[T // 2] = 0
        adapters = M.LoRAAdapters(torch.randn(1, 8, 64, device="cuda").to(BF16), torch.randn(1, 72, 8, device="cuda").to(BF16))
        got, h = M.lora_add(y, x, adapters, ids, save_for_backward=True)
        rest = ids < 0
        assert torch.equal(got.view(torch.int16)[rest], y.view(torch.int16)[rest]) and not h[rest].any()


def test_many_adapters():
    T, L = 5000, 1024
    g = torch.Generator("cuda").manual_seed(0)
    x, y = torch.randn(T, 128, device="cuda", generator=g).to(BF16), torch.randn(T, 80, device="cuda", generator=g).to(BF16)
    down, up = 0.1 * torch.randn(L, 16, 128, device="cuda", generator=g), torch.randn(L, 80, 16, device="cuda", generator=g)
    adapters = M.LoRAAdapters(down.to(BF16), up.to(BF16))
    ids = torch.randint(0, L, (T,), device="cuda", generator=g).to(torch.int32)
    ids[:3000] = 7                                                # and one of a few thousand tokens
    got, h = M.lora_add(y, x, adapters, ids, save_for_backward=True)
    for rows in (slice(0, 200), slice(2990, 3100), slice(4800, 5000)):
        assert torch.equal(got[rows], M.lora_add(y[rows], x[rows], adapters, ids[rows]))
    dx, ddown, dup = M.lora_add_backward(y, x, h, adapters, ids)
    used = ids.unique()
    want = OL.backward(values(y), values(x), values(h), values(adapters.tensors[0]), values(adapters.tensors[1]), np.ones(L), ids.cpu().numpy())
    for g_, w in ((ddown, want[1]), (dup, want[2])):
        assert np.linalg.norm(values(g_) - w) <= 2.0 ** -17 * np.linalg.norm(w)
    unused = torch.ones(L, dtype=torch.bool, device="cuda")
    unused[used.long()] = False
    assert not ddown[unused].any() and not dup[unused].any()
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T", [3, 700])
def test_a_block_with_adapters_and_a_balanced_router(T):
    """Router, its route and balance loss, a 4-bit projection with adapters, and the gradients of all of it."""
    H, E, k, L, R, N = 256, 32, 4, 3, 16, 320
    g = torch.Generator("cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, w_router = n(T, H).to(BF16), (0.05 * n(E, H)).to(BF16)
    w = (0.05 * n(N, H)).to(BF16)
    who = torch.randint(-1, L, (T,), device="cuda", generator=g).to(torch.int32)
    adapters = M.LoRAAdapters((n(L, R, H) / 16).to(BF16), (0.1 * n(L, N, R)).to(BF16), n(L).abs())
    weight = M.nvfp4_quantize_weight(w)
    _, _, logits = M.moe_router_topk(x, w_router, 1, with_logits=True)
    ids, p = M.moe_route_topk(logits, k)
    b = M.moe_balance_loss(logits, ids)
    y, h = M.lora_add(M.nvfp4_linear(x, weight), x, adapters, who, save_for_backward=True)
    # gradients: of the route's weights and of the loss into one buffer, of the projection into the adapters'
    dw, dy = n(T, k), n(T, N).to(BF16)
    dlogits = M.moe_route_topk_backward(logits, ids, dw)
    M.moe_balance_loss_backward(logits, k, b.counts, b.tokens, torch.full((1,), 0.01, device="cuda"), dlogits=dlogits)
    dx, ddown, dup = M.lora_add_backward(dy, x, h, adapters, who, dx=(dy.float() @ w.float()).to(BF16))
    assert M.nvfp4_get_device_error() == 0
    # the same in 64 bits
    l = values(logits)
    from oracle import route_topk as OR
    want = OR.backward(l, ids.cpu().numpy(), values(dw), "softmax", True, 1.0)
    _, counts, _, tokens = OB.loss(l, ids.cpu().numpy())
    want = want + OB.backward(l, k, counts, tokens, [0.01])[0]
    assert np.linalg.norm(values(dlogits) - want) <= 2e-5 * np.linalg.norm(want)
    base = Q.dequantize_rows(*Q.quantize_rows(x.float().cpu().numpy())) @ Q.dequantize_rows(*Q.quantize_rows(w.float().cpu().numpy())).T
    down, up, scale = (values(t) for t in adapters.tensors)
    want, want_h = OL.add(base, values(x), down, up, scale, who.cpu().numpy())
    # the projection's output is rounded to BF16, then the sum: half a step each
    assert np.linalg.norm(values(y) - want) <= 2 * 2.0 ** -8 * np.linalg.norm(want)
    grads = OL.backward(values(dy), values(x), want_h, down, up, scale, who.cpu().numpy())
    want = values(dy) @ values(w) + grads[0]
    assert np.linalg.norm(values(dx) - want) <= 2 * 2.0 ** -8 * np.linalg.norm(want) + 2.0 ** -8 * np.linalg.norm(values(dy) @ values(w))
    for got, w64 in ((ddown, grads[1]), (dup, grads[2])):
        assert np.linalg.norm(values(got) - w64) <= 2.0 ** -17 * np.linalg.norm(w64)


def test_the_example_block_with_adapters_and_a_balance_loss():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_block
    T, H, I, L, R = 200, 512, 256, 3, 8
    block = moe_block.MoEBlock(H=H, I=I, E=64, k=6, n_group=8, topk_group=4)
    g = torch.Generator("cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    block.add_adapters((0.1 * n(L, R, I)).to(BF16), (0.1 * n(L, H, R)).to(BF16), n(L))
    x, dout = n(T, H).to(BF16), n(T, H).to(BF16)
    who = torch.randint(-1, L, (T,), device="cuda", generator=g).to(torch.int32)
    cut = torch.tensor([0, 1, 120, T], dtype=torch.int32, device="cuda")
    plain = block.forward(x)
    y = block.forward(x, train=True, adapter_ids=who)
    assert torch.equal(y[who < 0], plain[who < 0]) and not torch.equal(y, plain)
    assert torch.equal(block.forward(x[7:8], adapter_ids=who[7:8]), y[7:8])
    block.forward(x, train=True, adapter_ids=who)
    dw_plain = block.backward(dout)[3]
    balance = block.balance_loss(cut)
    _, logits, ids = block.saved
    block.forward(x, train=True, adapter_ids=who)
    dw = block.backward(dout, balance, weight=50.0, seq_offsets=cut)[3]
    ddown, dup = block.adapter_gradients(dout)
    assert M.nvfp4_get_device_error() == 0
    loss, counts, _, tokens = OB.loss(values(logits), ids.cpu().numpy(), "sigmoid", offsets=cut.tolist())
    assert np.allclose(values(balance.loss), loss, rtol=1e-5, atol=0)
    want = OB.backward(values(logits), 6, counts, tokens, [50.0] * 3, "sigmoid", offsets=cut.tolist())[0].T @ values(x)
    # two gradients of 32-bit logits' gradients (2e-5 of their terms) and 32-bit products over 200 tokens
    assert np.linalg.norm(values(dw) - values(dw_plain) - want) <= 1e-4 * (np.linalg.norm(want) + np.linalg.norm(values(dw_plain)))
    act, h, _ = block.saved_shared
    down, up, scale = (values(t) for t in block.adapters.tensors)
    want = OL.backward(values(dout), values(act), values(h), down, up, scale, who.cpu().numpy())
    for got, w64 in ((ddown, want[1]), (dup, want[2])):
        assert np.linalg.norm(values(got) - w64) <= 2.0 ** -17 * np.linalg.norm(w64)
