"""GPU parity of moe_route_topk and its gradient against the FP64 oracle (oracle/route_topk.py).

Tolerances.  Scores are FP32: the exponential's argument l - m is off by 2^-24 |l - m| and expf by
2 ulp, a sum of E <= 1024 positive terms in a tree of depth <= 37 by 37 * 2^-24, the quotients by
one rounding each.  With |l - m| <= 30 that is below 75 * 2^-24 < 5e-6 relative: weights are held
to 5e-6 * w.  A gradient is held to 2e-5 times the sum of the magnitudes of the terms it is the
difference of (four such factors), plus its one rounding to the output's type.

Ids have to be equal where the order does not hang on a computed score's last bits: rows in which
two order values (with a bias) or two group scores lie within 2e-6 of each other without being
equal are left out of that comparison and are few.
"""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import route_topk as R

pytestmark = pytest.mark.gpu

W_REL = 5e-6
G_REL = 2e-5
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-38, torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def values(t):
    return t.detach().cpu().double().numpy()


def make(T, E, dtype=torch.float32, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed + 31 * T + E)
    return (spread * torch.randn(T, E, generator=g)).to(dtype).cuda()


def decided(l, k, score, bias, n_group, topk_group, group_score):
    """Rows whose ids no rounding of the scores can change: of the order values, the k + 1 that come
    first in the groups kept are looked at, of the group scores all."""
    ok = np.ones(l.shape[0], bool)

    def apart(v):
        v = -np.sort(-v, axis=1)
        with np.errstate(invalid="ignore"):
            gap = v[:, :-1] - v[:, 1:]
        return ~((gap > 0) & (gap < 2e-6)).any(1)

    o = R.order_values(l, score, bias)
    if n_group > 1 and (bias is not None or group_score == "top2"):
        gs = R.group_scores(l, score, bias, n_group, group_score)
        ok &= apart(gs)
        kept = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1) < topk_group
        o = np.where(np.repeat(kept, l.shape[1] // n_group, axis=1), o, -np.inf)
    if bias is not None:
        ok &= apart(-np.sort(-o, axis=1)[:, :k + 1])
    return ok


def check(logits, k, least=0.5, **kw):
    bias = kw.pop("bias", None)
    dev_bias = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids, w = M.moe_route_topk(logits, k, bias=dev_bias, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    ids, w = ids.cpu().numpy(), values(w)
    l = values(logits)
    b64 = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    want_ids, _ = R.route(l, k, bias=b64, **kw)
    ok = decided(l, k, kw.get("score", "softmax"), b64, kw.get("n_group", 1), kw.get("topk_group", 1),
                 kw.get("group_score", "max"))
    assert ok.mean() >= least
    assert np.array_equal(ids[ok], want_ids[ok])
    for row in ids:
        assert len(set(row)) == k and 0 <= row.min() and row.max() < l.shape[1]
    want = R.weights(l, ids, kw.get("score", "softmax"), kw.get("renormalize", True), kw.get("scale", 1.0))
    assert np.all(np.abs(w - want) <= W_REL * np.abs(want) + 1e-30), np.abs(w - want).max()
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 5, 5), (33, 31, 4), (9, 32, 32), (65, 33, 3), (130, 100, 8),
                                   (17, 128, 8), (40, 250, 6), (12, 256, 32), (21, 511, 10), (5, 1000, 12),
                                   (9, 1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_shapes(T, E, k, score, renorm):
    check(make(T, E), k, score=score, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E,k", [(8, 3), (60, 4), (128, 8), (1024, 16)])
def test_types(dtype, E, k):
    check(make(50, E, dtype), k)                             # equal logits are common: lower id first
    check(make(50, E, dtype), k, score="sigmoid", renormalize=False)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(16, 2, 1, 8), (64, 8, 3, 6), (256, 8, 4, 8), (60, 5, 2, 7),
                                                    (12, 12, 5, 4), (32, 32, 32, 32), (1024, 32, 2, 20), (96, 4, 4, 9)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score,with_bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True),
                                             ("softmax", True)])
def test_groups(E, n_group, topk_group, k, group_score, score, with_bias):
    bias = 0.05 * np.random.default_rng(E).standard_normal(E).astype(np.float32) if with_bias else None
    # 1024 softmax scores of mean 1/1024 lie close together: nearly every row has a pair within 2e-6
    check(make(70, E, seed=k), k, least=0.0 if E == 1024 and with_bias else 0.5, score=score, bias=bias,
          n_group=n_group, topk_group=topk_group, group_score=group_score)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(248, 8, 4, 8), (136, 8, 3, 9), (200, 2, 1, 8), (80, 16, 3, 4),
                                                    (93, 31, 7, 5), (510, 30, 4, 11), (29, 29, 9, 9), (1023, 11, 2, 6)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_groups_of_any_size(E, n_group, topk_group, k, group_score, dtype):
    bias = 0.05 * np.random.default_rng(E).standard_normal(E).astype(np.float32)
    for b in (None, bias):
        # of hundreds of scores one pair in most rows lies within 2e-6 (BF16 logits: also of equal scores plus a bias)
        check(make(70, E, dtype, seed=k), k, least=0.5 if b is None and group_score == "max" else 0.0, score="sigmoid", bias=b,
              n_group=n_group, topk_group=topk_group, group_score=group_score)


def test_ties_take_the_lower_id():
    l = torch.zeros((3, 64), device="cuda")
    ids, w = M.moe_route_topk(l, 5)
    assert ids.cpu().tolist() == [[0, 1, 2, 3, 4]] * 3 and torch.all(w == 0.2)
    l[:, 40] = 1.0
    l[:, 50] = 1.0
    l[:, 9] = -0.0                                           # equal to +0
    ids, _ = M.moe_route_topk(l, 4)
    assert ids.cpu().tolist() == [[40, 50, 0, 1]] * 3
    ids, _ = M.moe_route_topk(l * 0, 4, n_group=8, topk_group=2, group_score="top2", score="sigmoid",
                              bias=torch.zeros(64, device="cuda"))
    assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_experts(dtype, score, renorm):
    l = make(40, 48, dtype)
    inf = float("inf")
    l[0] = -inf                                              # nothing left
    l[1] = -inf
    l[1, 7] = 0.5                                            # one left, fewer than k
    l[2, ::2] = -inf
    l[3] = torch.finfo(dtype).min                            # the type's lowest value everywhere: no mask
    l[4, 5:] = torch.finfo(dtype).min
    l[5, 30:] = -inf
    bias = 0.02 * np.random.default_rng(1).standard_normal(48)
    for kw in (dict(), dict(bias=bias), dict(n_group=6, topk_group=2), dict(n_group=6, topk_group=2, group_score="top2"),
               dict(n_group=6, topk_group=3, group_score="top2", bias=bias)):
        ids, w = check(l, 6, score=score, renormalize=renorm, **kw)
        assert np.all(w[0] == 0.0) and np.isfinite(w).all()
        if "n_group" not in kw:
            assert ids[0].tolist() == [0, 1, 2, 3, 4, 5] and ids[1, 0] == 7
    assert M.nvfp4_get_device_error() == 0                   # -inf is a mask, not an error


def test_nan_and_infinite_logits_are_reported():
    l = make(4, 32)
    l[1, 3] = float("nan")
    ids, w = M.moe_route_topk(l, 4)
    assert M.nvfp4_get_device_error() == 6                   # NVFP4_ERR_NONFINITE
    assert 3 not in ids[1].tolist() and bool(torch.isfinite(w).all())
    l = make(4, 32)
    l[2, 9] = float("inf")
    l[2, 11] = float("inf")
    ids, w = M.moe_route_topk(l, 4)
    assert M.nvfp4_get_device_error() == 6
    assert ids[2, :2].tolist() == [9, 11] and w[2].tolist() == [0.5, 0.5, 0.0, 0.0]


def test_extreme_logits():
    l = make(20, 64, spread=1.0) * 1e4                       # differences far beyond the exponential's range
    for score in ("softmax", "sigmoid"):
        ids, w = M.moe_route_topk(l, 6, score=score)
        assert bool(torch.isfinite(w).all())
        want, _ = R.route(values(l), 6, score=score)
        assert np.array_equal(ids.cpu().numpy(), want)       # by logits: saturated scores do not tie


def test_bias_minus_infinity_is_chosen_last():
    l = make(10, 16)
    b = np.zeros(16, np.float32)
    b[[0, 5]] = -np.inf
    ids, w = check(l, 16, bias=b, score="sigmoid")
    assert ids[:, -2:].tolist() == [[0, 5]] * 10 and (w > 0).all()


def test_row_strides_and_empty_batches():
    big = make(33, 300)
    for view in (big[:, 10:138], big[::2, :128], big[:, :1]):
        a = M.moe_route_topk(view, min(8, view.shape[1]))
        b = M.moe_route_topk(view.contiguous(), min(8, view.shape[1]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        dw = torch.randn(view.shape[0], a[0].shape[1], device="cuda")
        for score in ("softmax", "sigmoid"):
            for r in (True, False):
                assert torch.equal(M.moe_route_topk_backward(view, a[0], dw, score=score, renormalize=r),
                                   M.moe_route_topk_backward(view.contiguous(), a[0], dw, score=score, renormalize=r))
    ids, w = M.moe_route_topk(big[:0], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert M.moe_route_topk_backward(big[:0], ids, w).shape == (0, 300)


def test_batch_invariance():
    l = make(300, 256)
    b = 0.02 * torch.randn(256, device="cuda")
    kw = dict(score="sigmoid", bias=b, n_group=8, topk_group=4, group_score="top2", scale=2.5)
    ids, w = M.moe_route_topk(l, 8, **kw)
    dl = M.moe_route_topk_backward(l, ids, w, score="sigmoid", scale=2.5)
    for lo, hi in ((0, 1), (7, 8), (299, 300), (3, 100), (128, 300)):
        i2, w2 = M.moe_route_topk(l[lo:hi], 8, **kw)
        assert torch.equal(i2, ids[lo:hi]) and torch.equal(w2, w[lo:hi])
        assert torch.equal(M.moe_route_topk_backward(l[lo:hi], i2, w2, score="sigmoid", scale=2.5), dl[lo:hi])


def gradient_bound(l, ids, dw, score, renorm, scale, dtype):
    """Magnitudes of the terms each gradient is the difference of."""
    T, E = l.shape
    i = ids.astype(np.int64)
    w1 = R.weights(l, ids, score, renorm, 1.0)
    g = np.abs(dw * scale)
    dot = (g * w1).sum(1, keepdims=True)
    own = np.zeros((T, E))
    if score == "softmax" and not renorm:
        s = R.scores(l, score)
        np.put_along_axis(own, i, g, 1)
        terms = s * (own + dot)
    else:
        np.put_along_axis(own, i, w1 * (g + (dot if renorm else 0.0)), 1)
        terms = own
    return terms


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (33, 31, 4), (9, 32, 32), (65, 100, 8), (17, 128, 8), (40, 250, 6),
                                   (7, 1024, 32)])
def test_gradient(dtype, score, renorm, T, E, k):
    l = make(T, E, dtype, seed=5)
    if T > 2:
        l[1, : E // 2] = -float("inf")
        l[2] = -float("inf")
    ids, _ = M.moe_route_topk(l, k, score=score, renormalize=renorm)
    dw = torch.randn(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    got = M.moe_route_topk_backward(l, ids, dw, score=score, renormalize=renorm, scale=2.5)
    assert got.dtype == dtype and got.shape == l.shape
    l64, i, d64 = values(l), ids.cpu().numpy(), values(dw)
    want = R.backward(l64, i, d64, score, renorm, 2.5)
    tol = G_REL * gradient_bound(l64, i, d64, score, renorm, 2.5, dtype) + UNIT[dtype] * np.abs(want) + TINY[dtype]
    assert np.all(np.abs(values(got) - want) <= tol)
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(41, 251, 6), (9, 127, 8), (5, 501, 12), (33, 63, 5), (3, 1023, 32), (6, 254, 20)])
def test_gradient_of_odd_rows(dtype, renorm, T, E, k):
    l = make(T, E, dtype, seed=9)
    l[1, 3: E // 2] = -float("inf")
    ids, _ = M.moe_route_topk(l, k, renormalize=renorm)
    dw = torch.randn(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    got = M.moe_route_topk_backward(l, ids, dw, renormalize=renorm)
    l64, i, d64 = values(l), ids.cpu().numpy(), values(dw)
    want = R.backward(l64, i, d64, "softmax", renorm, 1.0)
    tol = G_REL * gradient_bound(l64, i, d64, "softmax", renorm, 1.0, dtype) + UNIT[dtype] * np.abs(want) + TINY[dtype]
    assert np.all(np.abs(values(got) - want) <= tol)
    # into rows of another pitch on any boundary, nothing beside them written
    p = M.moe_route_params(0, k, 1, 1, 0, 1 if renorm else 0, 1.0)
    for lo, pitch in ((0, E + 5), (1, E + 1), (2, E + 2), (3, E + 4), (8, E + 24 - E % 8)):
        out = torch.full((T, pitch), 7.0, dtype=dtype, device="cuda")
        status = M.lib().moe_route_topk_backward(l.data_ptr(), M._TYPES[dtype], T, E, E, p, ids.data_ptr(), dw.data_ptr(),
                                                 out[:, lo:].data_ptr(), pitch, torch.cuda.current_stream().cuda_stream)
        assert status == 0 and torch.equal(out[:, lo:lo + E], got)
        assert bool((out[:, :lo] == 7.0).all()) and bool((out[:, lo + E:] == 7.0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences_of_the_kernel(score, renorm):
    # central differences of FP32 weights with h = 2^-6: the third derivatives are below 1 and the
    # weights' error below 1e-6, so |difference - gradient| <= k max|dw| (h^2 / 6 + 1e-6 / h)
    h, k, E = 2.0 ** -6, 4, 12
    l = make(8, E, seed=9)
    ids, _ = M.moe_route_topk(l, k, score=score, renormalize=renorm)
    dw = torch.randn(8, k, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    got = values(M.moe_route_topk_backward(l, ids, dw, score=score, renormalize=renorm))
    bound = k * float(dw.abs().max()) * (h * h / 6 + 1e-6 / h)

    def total(x):
        # the weights of the same experts: all E are chosen and the fixed ids' entries taken
        if renorm:
            x = torch.gather(x, 1, ids.long())
        i2, w2 = M.moe_route_topk(x.contiguous(), x.shape[1], score=score, renormalize=renorm)
        w = torch.zeros_like(x).scatter_(1, i2.long(), w2)
        if not renorm:
            w = torch.gather(w, 1, ids.long())
        return values((w * dw).sum(1))

    for e in range(E):
        up, dn = l.clone(), l.clone()
        up[:, e] += h
        dn[:, e] -= h
        diff = (total(up) - total(dn)) / (2 * h)
        assert np.all(np.abs(diff - got[:, e]) <= bound), e


def test_gradient_reports_bad_ids():
    l = make(4, 16)
    ids, w = M.moe_route_topk(l, 2)
    bad = ids.clone()
    bad[1, 0], bad[2, 1] = 16, -1
    got = M.moe_route_topk_backward(l, bad, torch.ones_like(w))
    assert M.nvfp4_get_device_error() == 5                   # NVFP4_ERR_BAD_EXPERT_ID
    assert bool(torch.isfinite(got).all())
    good = M.moe_route_topk_backward(l, ids, torch.ones_like(w))
    assert torch.equal(got[[0, 3]], good[[0, 3]])


def test_another_stream():
    l = make(500, 128)
    want = M.moe_route_topk(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.moe_route_topk(l, 8, stream=s)
    dl = M.moe_route_topk_backward(l, got[0], got[1], stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(dl, M.moe_route_topk_backward(l, *want))


def test_large_batch_offsets():
    # the last rows of a batch whose element offsets pass 2^31
    T, E = (1 << 31) // 512 + 5, 512
    l = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = make(5, E, torch.bfloat16)
    l[-5:] = tail
    ids, w = M.moe_route_topk(l, 8)
    i2, w2 = M.moe_route_topk(tail, 8)
    assert torch.equal(ids[-5:], i2) and torch.equal(w[-5:], w2)
    dw = torch.randn(T, 8, device="cuda")
    dl = M.moe_route_topk_backward(l, ids, dw)
    assert torch.equal(dl[-5:], M.moe_route_topk_backward(tail, i2, dw[-5:].contiguous()))
