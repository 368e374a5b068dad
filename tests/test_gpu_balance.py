"""GPU parity of moe_balance_loss and its gradient against the FP64 oracle (oracle/balance.py).

Tolerances, with u = 2^-24.  A probability is within 75 u of its value (the exponential's argument off by u |l - m|,
|l - m| <= 30, expf by 2 ulp, a sum of E <= 1024 positive terms in a tree of depth <= 37, the quotients by one rounding
each: the bound of the routing's tests).  Means add n <= T positive terms, in a chain of at most T / 64 + 2 for the rows of
one lane and a tree of at most 40 joins beside it, and divide: (T / 64 + 43) u more.  The loss is a sum of E positive
terms of them, in a tree of at most 40, times a factor of three roundings: 43 u more.  A gradient is the difference of terms that
carry a probability or two each (150 u), the factors of g (4 u) and a tree (40 u): 200 u < 2e-5 of the sum of their
magnitudes, and half a step of the type."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import balance as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
G_REL = 2e-5
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-38, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}     # half the smallest step


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def values(t):
    return t.detach().cpu().double().numpy()


def make(T, E, k, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * T + E)
    l = (1.5 * torch.randn(T, E, generator=g)).to(dtype)
    ids = torch.randn(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    return l.cuda(), ids.cuda()


def cuts(T, S, seed):
    """S sequences of uneven lengths, some empty, rows in front of the first and behind the last."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, T + 1, (S + 1,), generator=g).sort().values.to(torch.int32)


def check(l, ids, score="softmax", mask=None, offsets=None, out_unit=None):
    kw = dict(score=score, mask=None if mask is None else mask.cuda(), seq_offsets=None if offsets is None else offsets.cuda())
    b = M.moe_balance_loss(l, ids, **kw)
    T, E = l.shape
    want = O.loss(values(l), ids.cpu().numpy(), score, None if mask is None else mask.numpy(),
                  None if offsets is None else offsets.numpy())
    assert [t.dtype for t in b] == [torch.float32, torch.int32, torch.float32, torch.int32]
    assert np.array_equal(b.counts.cpu().numpy(), want[1]) and np.array_equal(b.tokens.cpu().numpy(), want[3])
    p_rel = (75 + T / 64 + 43) * U
    assert np.all(np.abs(values(b.probs) - want[2]) <= p_rel * want[2] + 1e-37)
    assert np.all(np.abs(values(b.loss) - want[0]) <= (p_rel + 43 * U) * want[0])
    S = b.loss.shape[0]
    dloss = torch.randn(S, generator=torch.Generator().manual_seed(T)).cuda()
    grad = lambda **more: M.moe_balance_loss_backward(l, ids.shape[1], b.counts, b.tokens, dloss, **kw, **more)  # noqa: E731
    d = grad()
    assert d.dtype == l.dtype and d.shape == l.shape
    want_d, size = O.backward(values(l), ids.shape[1], want[1], want[3], values(dloss), score,
                              None if mask is None else mask.numpy(), None if offsets is None else offsets.numpy())
    tol = G_REL * size + HALF[l.dtype] * np.abs(want_d) + TINY[l.dtype]
    assert np.all(np.abs(values(d) - want_d) <= tol)
    assert not values(d)[size.sum(1) == 0].any()
    # added to what is there, in FP32 with one rounding
    was = torch.randn(l.shape, generator=torch.Generator().manual_seed(1)).to(l.dtype).cuda()
    got = grad(dlogits=was.clone())
    total = values(was) + want_d
    assert np.all(np.abs(values(got) - total) <= G_REL * size + (HALF[l.dtype] + U) * np.abs(total) + TINY[l.dtype] + U * np.abs(want_d))
    still = size.sum(1) == 0
    assert torch.equal(got.cpu()[still], was.cpu()[still])
    return b, d


SIZES = [(1, 1, 1), (1, 8, 2), (3, 128, 8), (8, 7, 3), (33, 31, 4), (65, 33, 3), (130, 100, 8), (9, 250, 6), (70, 256, 32),
         (21, 511, 10), (5, 1000, 12), (66, 1024, 8), (700, 60, 4)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("S", [None, 1, 5])
def test_sizes(T, E, k, score, S):
    l, ids = make(T, E, k)
    check(l, ids, score, None if S is None else torch.rand(T, generator=torch.Generator().manual_seed(S)) < 0.7,
          None if S is None else cuts(T, S, T + S))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", [(40, 8, 3), (100, 128, 8), (50, 250, 4), (33, 1024, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_types(dtype, T, E, k, score):
    l, ids = make(T, E, k, dtype)
    check(l, ids, score, torch.arange(T) % 3 != 0, cuts(T, 3, E))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T,S", [(5000, 1), (5000, 3), (4099, 400), (300, 300), (2000, 2000), (64, 3000)])
def test_many_rows_and_sequences(T, S):
    l, ids = make(T, 64, 6)
    check(l, ids, "sigmoid", torch.rand(T, generator=torch.Generator().manual_seed(S)) < 0.9, cuts(T, S, S))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T,E,S", [(1024, 128, 1), (1025, 128, 1), (512, 256, 3), (513, 256, 3), (4096, 64, 4), (4097, 64, 4), (512, 128, 1),
                                   (513, 128, 7), (513, 128, 8), (4096, 128, 1), (4097, 128, 1), (512, 1000, 2), (525, 1000, 2),
                                   (2048, 256, 5), (900, 64, 64), (900, 64, 65), (4100, 96, 19), (4100, 96, 20),
                                   (4100, 96, 38), (4100, 96, 39), (4100, 96, 76), (4100, 96, 77), (3000, 96, 152), (3000, 96, 153)])
def test_where_the_ways_meet(T, E, S):
    """One kernel or two, and the sizes of the second one's clusters."""
    l, ids = make(T, E, 6)
    check(l, ids, "softmax", torch.rand(T, generator=torch.Generator().manual_seed(S)) < 0.9, None if S == 1 else cuts(T, S, S))
    if S > 1:                              # all the tokens in one of them
        one = torch.full((S + 1,), T, dtype=torch.int32)
        one[: S // 2 + 1] = 0
        check(l, ids, "sigmoid", None, one)
    assert M.nvfp4_get_device_error() == 0


def test_runs_of_empty_sequences():
    T, S = 3000, 300000
    l, ids = make(T, 8, 2)
    cut = torch.full((S + 1,), 1400, dtype=torch.int32)             # a quarter of a million empty ones between two rows
    cut[:1000] = torch.arange(1000)
    cut[260000:] = torch.arange(S + 1 - 260000).clamp(max=1500) + 1400
    b = M.moe_balance_loss(l, ids, seq_offsets=cut.cuda())
    tokens = cut.diff()
    assert torch.equal(b.tokens.cpu(), tokens)
    some = torch.cat([tokens.nonzero().flatten(), torch.tensor([1000, 200000, S - 1])])
    dloss = torch.ones(S).cuda()
    d = M.moe_balance_loss_backward(l, 2, b.counts, b.tokens, dloss, seq_offsets=cut.cuda())
    p = torch.softmax(l.double().cpu(), 1)
    for s in some[::97].tolist() + [999, 1000, 259999, 260000, S - 1]:
        rows = slice(int(cut[s]), int(cut[s + 1]))
        n = rows.stop - rows.start
        c = torch.bincount(ids[rows].flatten().cpu().long(), minlength=8)
        assert torch.equal(b.counts[s].cpu().long(), c)
        mean = p[rows].mean(0) if n else torch.zeros(8, dtype=torch.float64)
        want = (c * mean).sum() * 8 / (2 * n) if n else 0.0
        assert abs(float(b.loss[s]) - float(want)) <= 200 * U * float(want)
        if n:
            g = 8.0 * c / (2.0 * n * n)
            want = p[rows] * (g - (g * p[rows]).sum(1, keepdim=True))
            assert np.all(np.abs(values(d[rows]) - want.numpy()) <= G_REL * (p[rows] * (g + (g * p[rows]).sum(1, keepdim=True))).numpy() + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score):
    l, ids = make(50, 40, 4, seed=3)
    inf = float("inf")
    l[0] = -inf                                                   # nothing left
    l[1, ::2] = -inf
    l[2] = torch.finfo(torch.float32).min                         # a mask by the type's lowest value
    l[3, 5:] = torch.finfo(torch.float32).min
    l[4] = -400.0 - torch.arange(40)                              # sigmoids below FP32's range
    l[5] = 1e30
    check(l, ids, score)
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_logits(score, value):
    l, ids = make(20, 24, 3, seed=4)
    l[7, 3] = value
    l[7, 9] = value
    check(l, ids, score)                                          # NaN masks, +inf is the limit of large logits
    assert M.nvfp4_get_device_error() == 6
    # in a token that does not count they are nothing, nor are its ids
    mask = torch.ones(20, dtype=torch.bool)
    mask[7] = False
    ids[7] = 10 ** 9
    check(l, ids, score, mask)
    assert M.nvfp4_get_device_error() == 0
    assert not M.moe_balance_loss_backward(l, 3, torch.ones(1, 24, dtype=torch.int32, device="cuda"),
                                           torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda"),
                                           score=score, mask=mask.cuda())[7].any()


def test_bad_ids_are_reported_and_not_counted():
    l, ids = make(30, 16, 2, seed=5)
    ids[3, 1], ids[9, 0] = 16, -1
    b = M.moe_balance_loss(l, ids)
    assert M.nvfp4_get_device_error() == 5
    assert np.array_equal(b.counts.cpu().numpy(), O.loss(values(l), ids.cpu().numpy())[1]) and int(b.counts.sum()) == 58


def test_nothing_counts():
    l, ids = make(17, 32, 4)
    b, d = check(l, ids, mask=torch.zeros(17, dtype=torch.bool))
    assert not b.loss.any() and not d.any()
    b, d = check(l, ids, offsets=torch.full((4,), 17, dtype=torch.int32))
    assert not b.tokens.any() and not d.any()
    b = M.moe_balance_loss(l[:0], ids[:0], seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert not any(t.any() for t in b) and b.loss.shape == (2,)
    assert M.moe_balance_loss_backward(l[:0], 4, *b[1:4:2], torch.ones(2, device="cuda"),
                                       seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 32)


def test_offsets_outside_the_rows_stay_inside():
    # not what the call asks for: nothing outside the rows is read or written
    l, ids = make(40, 64, 4)
    for off in ([0, 100, 1 << 30], [-5, 3, 2], [50, 20, 10], [30, 10, 40]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        b = M.moe_balance_loss(l, ids, seq_offsets=off)
        M.moe_balance_loss_backward(l, 4, b.counts, b.tokens, b.loss, seq_offsets=off)
        assert int(b.tokens.max()) <= 40 and int(b.tokens.min()) >= 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_alignment(dtype):
    T, E, k = 70, 128, 5
    l, ids = make(T, E, k, dtype)
    want_b, want_d = check(l, ids, "sigmoid")
    for left, pitch in ((0, 136), (3, 140), (1, 129), (8, 144)):
        wide = torch.full((T, pitch), float("nan"), dtype=dtype, device="cuda")
        v = wide[:, left:left + E]
        v.copy_(l)
        b = M.moe_balance_loss(v, ids, score="sigmoid")
        assert torch.equal(b.counts, want_b.counts)
        assert np.all(np.abs(values(b.probs) - values(want_b.probs)) <= 300 * U * values(want_b.probs))
        out = torch.full((T, pitch), 7.0, dtype=dtype, device="cuda")
        o = out[:, left:left + E]
        o.zero_()
        M.moe_balance_loss_backward(v, k, b.counts, b.tokens, torch.ones(1, device="cuda"), score="sigmoid", dlogits=o)
        assert (out[:, :left] == 7).all() and (out[:, left + E:] == 7).all()
        one = M.moe_balance_loss_backward(l, k, b.counts, b.tokens, torch.ones(1, device="cuda"), score="sigmoid")
        assert np.all(np.abs(values(o) - values(one)) <= 2 * G_REL * np.abs(values(one)).max() + HALF[dtype] * np.abs(values(one)))
    assert M.nvfp4_get_device_error() == 0


def test_counts_of_a_larger_batch():
    # two halves with the sums of their counts and tokens give the gradient of the whole
    l, ids = make(120, 48, 6)
    whole = M.moe_balance_loss(l, ids)
    halves = [M.moe_balance_loss(l[a:a + 60], ids[a:a + 60]) for a in (0, 60)]
    counts, tokens = sum(h.counts for h in halves), sum(h.tokens for h in halves)
    assert torch.equal(counts, whole.counts) and torch.equal(tokens, whole.tokens)
    g = torch.full((1,), 0.3, device="cuda")
    want = M.moe_balance_loss_backward(l, 6, whole.counts, whole.tokens, g)
    got = torch.cat([M.moe_balance_loss_backward(l[a:a + 60], 6, counts, tokens, g) for a in (0, 60)])
    assert torch.equal(got, want)


def test_same_call_same_bits():
    l, ids = make(3000, 128, 8)
    off = cuts(3000, 7, 1).cuda()
    a, b = (M.moe_balance_loss(l, ids, seq_offsets=off) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
