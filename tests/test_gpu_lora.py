"""GPU parity of lora_add and lora_add_backward against the FP64 oracle (oracle/lora.py).

Tolerances.  Products of 16-bit values are exact in FP32; an m16n8k16 step adds 16 of them to an accumulator with an error
of at most 2^-22 of the magnitudes it adds.  h: chains of n = ceil(K / 1024) steps, then 16 FP32 additions: (n + 4) 2^-22
of sum |x| |A|.  The second product takes h to 2^-16 (two BF16 terms: each leaves 2^-8), 2^-24 (three) or 2^-22 (two FP16
terms, scaled by the row's largest), in R / 16 steps a term: (3 R / 16 + 1) 2^-22 of sum |h| |B|; then y is added in
FP32 (2^-24 of the sum) and the output rounded (half a step of its type).  Gradients of the adapters sum over tokens: three
terms to a token's step, at most 3 (T / 16 + 1) steps and 8 + 2 additions, and dh's or h's own error."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import lora as O

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 1e-38, BF16: 1e-38, F16: 2.0 ** -25}
STEP = 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def values(t):
    return t.detach().cpu().double().numpy()


class Case:
    def __init__(self, T, K, N, R, L, dtype=BF16, out=BF16, seed=0, none=0.15, order="random", scaled=True):
        g = torch.Generator().manual_seed(seed + T + 3 * K + 5 * N + R)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x, self.y, self.dy = n(T, K).to(dtype), n(T, N).to(out), (0.1 * n(T, N)).to(dtype)
        self.down, self.up = (n(L, R, K) / K ** 0.5).to(dtype), (0.1 * n(L, N, R)).to(dtype)
        self.scale = 0.5 + torch.rand(L, generator=g) if scaled else None
        ids = (torch.rand(T, generator=g) ** 2 * L).to(torch.int32).clamp(max=L - 1)
        ids[torch.rand(T, generator=g) < none] = -1
        self.ids = ids.sort().values if order == "sorted" else ids
        self.T, self.K, self.N, self.R, self.L = T, K, N, R, L
        for name in ("x", "y", "dy", "down", "up", "scale", "ids"):
            v = getattr(self, name)
            setattr(self, name, None if v is None else v.cuda())
        self.adapters = M.LoRAAdapters(self.down, self.up, self.scale)

    def scales(self):
        return np.ones(self.L) if self.scale is None else values(self.scale)

    def matrices(self):
        return values(self.down), values(self.up), self.scales(), self.ids.cpu().numpy()

    def forward_bounds(self, dtype, out):
        """(out, h, tolerance of out, of h)."""
        x, (down, up, scale, ids) = values(self.x), self.matrices()
        want, h = O.add(values(self.y), x, down, up, scale, ids)
        zero = np.zeros_like(values(self.y))
        h_tol = ((self.K + 1023) // 1024 + 4) * STEP * O.add(zero, abs(x), abs(down), abs(up), scale, ids)[1]
        return want, h, self.second(zero, h, h_tol, up, ids, dtype, out, want), h_tol

    def second(self, zero, h, h_tol, up, ids, dtype, out, want):
        keep = 2.0 ** -22 if dtype == F16 else 2.0 ** -24 if out == F32 else 2.0 ** -16
        tol = zero.copy()
        for a in range(self.L):
            rows = ids == a
            each = h_tol[rows] + (keep + (3 * self.R / 16 + 4) * STEP) * abs(h[rows])
            if dtype == F16 and rows.any():
                each = each + 2.0 ** -36 * abs(h[rows]).max(1, keepdims=True)
            tol[rows] = self.scales()[a] * (each @ abs(up[a]).T)
        return tol * 1.01 + (HALF[out] + 2.0 ** -23) * (abs(want) + tol) + TINY[out]


def check(c, dtype=BF16, out=BF16, **kw):
    got, h = M.lora_add(c.y, c.x, c.adapters, c.ids, save_for_backward=True, **kw)
    assert got.dtype == out and h.dtype == F32
    want, want_h, tol, h_tol = c.forward_bounds(dtype, out)
    assert np.all(np.abs(values(h) - want_h) <= h_tol + 1e-37)
    assert np.all(np.abs(values(got) - want) <= tol)
    none = (c.ids < 0) | (c.ids >= c.L)
    assert torch.equal(got[none], c.y[none])
    assert torch.equal(M.lora_add(c.y, c.x, c.adapters, c.ids), got)
    return got, h


FEW = [(1, 8, 1, 8, 1), (1, 64, 33, 16, 3), (2, 1024, 512, 16, 1), (5, 128, 70, 24, 2), (16, 1032, 96, 8, 5),
       (17, 2080, 1999, 16, 20), (40, 4096, 64, 64, 4), (33, 5000, 300, 32, 9), (9, 8200, 100, 128, 2), (64, 520, 600, 72, 64),
       (256, 136, 130, 128, 40), (200, 256, 2100, 16, 2), (255, 96, 40, 40, 300),
       (20, 64, 5000, 16, 3), (3, 64, 4100, 104, 2)]
SORTED = [(257, 256, 100, 16, 6), (300, 1024, 257, 40, 1), (1000, 136, 72, 16, 1024), (700, 2048, 90, 128, 3)]
MANY = [(3025, 136, 72, 16, 3), (1300, 2048, 200, 64, 7), (1100, 1088, 513, 128, 2), (1500, 8, 1, 8, 1), (2000, 4104, 70, 24, 9),
        (1200, 1032, 1000, 32, 200)]


@pytest.mark.parametrize("shape", FEW + SORTED + MANY)
def test_sizes(shape):
    check(Case(*shape))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("shape", [(3, 256, 129, 16, 2), (77, 2080, 1999, 8, 20), (300, 520, 100, 48, 5), (1100, 2048, 130, 64, 3),
                                   (1030, 264, 72, 128, 2)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_types(shape, dtype, out):
    check(Case(*shape, dtype=dtype, out=out), dtype, out)
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T", [7, 300, 1500])
def test_without_scales_and_in_place(T):
    c = Case(T, 264, 203, 24, 3, scaled=False)
    got, _ = check(c)
    y = c.y.clone()
    assert M.lora_add(y, c.x, c.adapters, c.ids, out=y) is y and torch.equal(y, got)


@pytest.mark.parametrize("T", [9, 400, 1300])
@pytest.mark.parametrize("ids", ["none", "one", "last"])
def test_one_adapter_or_none(T, ids):
    c = Case(T, 128, 96, 16, 5)
    c.ids.fill_({"none": -1, "one": 0, "last": 4}[ids])
    got, h = check(c)
    if ids == "none":
        assert torch.equal(got, c.y) and not h.any()


def test_a_row_does_not_depend_on_the_batch():
    for dtype, out, R in ((BF16, BF16, 16), (BF16, F32, 64), (F16, F16, 128), (BF16, BF16, 24)):
        c = Case(3000, 2056, 321, R, 6, dtype, out, seed=R)
        whole, h = M.lora_add(c.y, c.x, c.adapters, c.ids, save_for_backward=True)
        for n in (1, 5, 16, 100, 256, 257, 1024, 1025, 2500):
            at = torch.randperm(3000, generator=torch.Generator().manual_seed(n))[:n].cuda()
            got, got_h = M.lora_add(c.y[at].contiguous(), c.x[at].contiguous(), c.adapters, c.ids[at].contiguous(), save_for_backward=True)
            assert torch.equal(got, whole[at]) and torch.equal(got_h, h[at]), (dtype, R, n)


@pytest.mark.parametrize("T", [30, 300, 1200])
def test_strides_and_alignment(T):
    c = Case(T, 256, 96, 16, 3)
    want, want_h = check(c)
    for x_pitch, y_left, y_pitch, o_left, o_pitch in ((264, 0, 104, 8, 112), (512, 1, 97, 0, 96), (256, 3, 100, 5, 101)):
        x = torch.full((T, x_pitch), float("nan"), dtype=BF16, device="cuda")
        y = torch.full((T, y_pitch), float("nan"), dtype=BF16, device="cuda")
        o = torch.full((T, o_pitch), 7.0, dtype=BF16, device="cuda")
        x[:, :256], y[:, y_left:y_left + 96] = c.x, c.y
        got = M.lora_add(y[:, y_left:y_left + 96], x[:, :256], c.adapters, c.ids, out=o[:, o_left:o_left + 96])
        assert torch.equal(got, want)
        assert (o[:, :o_left] == 7).all() and (o[:, o_left + 96:] == 7).all()


@pytest.mark.parametrize("T", [20, 500, 1100])
def test_bad_ids_are_reported(T):
    c = Case(T, 64, 40, 8, 3)
    c.ids[T // 2], c.ids[1] = 3, 2 ** 31 - 1
    check(c)
    assert M.nvfp4_get_device_error() == 5


@pytest.mark.parametrize("T", [20, 500, 1100])
def test_nonfinite_rows_stay_theirs(T):
    c = Case(T, 64, 40, 8, 2, none=0.0)
    want = M.lora_add(c.y, c.x, c.adapters, c.ids)
    c.x[3, 5], c.x[7, 0] = float("nan"), float("inf")
    got = M.lora_add(c.y, c.x, c.adapters, c.ids)
    assert got[3].isnan().all() and not got[7].isfinite().any()
    rest = torch.ones(T, dtype=torch.bool)
    rest[[3, 7]] = False
    assert torch.equal(got.cpu()[rest], want.cpu()[rest])


@pytest.mark.parametrize("T", [20, 1100])
@pytest.mark.parametrize("size", [2.0 ** -18, 2.0 ** 6])
def test_fp16_h_of_any_size(T, size):
    # h far below and above FP16's range
    c = Case(T, 512, 64, 16, 2, F16, F32)
    c.x.mul_(size)
    c.down.mul_(2.0 ** -5 if size < 1 else 2.0 ** 13)
    c.y.zero_()
    check(c, F16, F32)
    _, h = M.lora_add(c.y, c.x, c.adapters, c.ids, save_for_backward=True)
    assert float(h.abs().max()) > 70000 or size < 1


def test_rows_past_32_bits():
    T, pitch = 600, 1 << 22                                       # 5 GB each
    c = Case(T, 64, 48, 8, 2)
    want = M.lora_add(c.y, c.x, c.adapters, c.ids)
    x = torch.empty((T - 1) * pitch + 64, dtype=BF16, device="cuda").as_strided((T, 64), (pitch, 1))
    y = torch.empty((T - 1) * pitch + 48, dtype=BF16, device="cuda").as_strided((T, 48), (pitch, 1))
    x.copy_(c.x)
    y.copy_(c.y)
    assert torch.equal(M.lora_add(y, x, c.adapters, c.ids), want)
    assert torch.equal(M.lora_add(y, x, c.adapters, c.ids, out=y), want)


def test_nothing_to_do():
    c = Case(4, 64, 40, 8, 3)
    assert M.lora_add(c.y[:0], c.x[:0], c.adapters, c.ids[:0]).shape == (0, 40)
    dx, ddown, dup = M.lora_add_backward(c.dy[:0], c.x[:0], torch.empty(0, 8, device="cuda"), c.adapters, c.ids[:0])
    assert dx.shape == (0, 64) and not ddown.any() and not dup.any() and ddown.shape == (3, 8, 64) and dup.shape == (3, 40, 8)


def check_backward(c, dx_type=BF16):
    T, N, K, R = c.T, c.N, c.K, c.R
    _, h = M.lora_add(c.y, c.x, c.adapters, c.ids, save_for_backward=True)
    dx, ddown, dup = M.lora_add_backward(c.dy, c.x, h, c.adapters, c.ids)
    assert dx.dtype == BF16 and ddown.dtype == dup.dtype == F32
    x, dy, hv, (down, up, scale, ids) = values(c.x), values(c.dy), values(h), c.matrices()
    want_dx, want_ddown, want_dup, dh = O.backward(dy, x, hv, down, up, scale, ids)
    zero = np.zeros_like(x)
    dh_tol = ((N + 1023) // 1024 + 5) * STEP * O.backward(abs(dy), abs(x), abs(hv), abs(down), abs(up), scale, ids)[3]

    def dx_tol(out, total):
        keep = 2.0 ** -24 if out == F32 else 2.0 ** -16
        tol = zero.copy()
        for a in range(c.L):
            rows = ids == a
            tol[rows] = (dh_tol[rows] + (keep + (3 * R / 16 + 4) * STEP) * abs(dh[rows])) @ abs(down[a])
        return tol * 1.01 + (HALF[out] + 2.0 ** -23) * (abs(total) + tol) + TINY[out]

    assert np.all(np.abs(values(dx) - want_dx) <= dx_tol(BF16, want_dx))
    was = torch.randn(T, K, generator=torch.Generator().manual_seed(K)).to(dx_type).cuda()
    got, again_down, again_up = M.lora_add_backward(c.dy, c.x, h, c.adapters, c.ids, dx=was.clone())
    assert np.all(np.abs(values(got) - (values(was) + want_dx)) <= dx_tol(dx_type, values(was) + want_dx))
    none = (c.ids < 0) | (c.ids >= c.L)
    assert torch.equal(got[none], was[none]) and not dx[none].any()
    assert torch.equal(again_down, ddown) and torch.equal(again_up, dup)     # the same bits
    n = 3 * (T / 16 + 1) + 10
    size = O.backward(abs(dy), abs(x), abs(hv), abs(down), abs(up), scale, ids)
    for a in range(c.L):
        rows = ids == a
        tol = (dh_tol[rows] + (2.0 ** -24 + n * STEP) * abs(dh[rows])).T @ abs(x[rows])
        assert np.all(np.abs(values(ddown[a]) - want_ddown[a]) <= 1.01 * tol + 1e-37)
        tol = (2.0 ** -23 + n * STEP) * size[2][a]
        assert np.all(np.abs(values(dup[a]) - want_dup[a]) <= 1.01 * tol + 1e-37)
    return dx, ddown, dup


BACKWARD = [(1, 8, 1, 8, 1), (3, 64, 33, 16, 2), (100, 520, 130, 24, 4), (257, 1032, 257, 16, 300), (300, 2048, 768, 64, 1),
            (500, 264, 1999, 128, 3), (1024, 128, 136, 8, 5), (1300, 1088, 999, 40, 2), (1100, 136, 520, 128, 2), (2100, 512, 256, 64, 4),
            (1500, 256, 8, 32, 7), (1500, 8, 1100, 16, 1), (2, 3272, 268, 24, 4), (300, 4600, 70, 16, 2), (30, 5000, 33, 72, 2)]


@pytest.mark.parametrize("shape", BACKWARD)
@pytest.mark.parametrize("dx_type", [BF16, F32, F16])
def test_backward(shape, dx_type):
    check_backward(Case(*shape), dx_type)
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T", [40, 1200])
@pytest.mark.parametrize("ids", ["none", "one", "sorted"])
def test_backward_of_one_adapter_or_none(T, ids):
    c = Case(T, 256, 200, 16, 3, order="sorted" if ids == "sorted" else "random", scaled=False)
    if ids != "sorted":
        c.ids.fill_(-1 if ids == "none" else 2)
    dx, ddown, dup = check_backward(c)
    if ids == "none":
        assert not dx.any() and not ddown.any() and not dup.any()


@pytest.mark.parametrize("T", [40, 1200])
def test_backward_bad_ids(T):
    c = Case(T, 64, 40, 8, 3)
    c.ids[5] = 3
    check_backward(c)
    assert M.nvfp4_get_device_error() == 5


@pytest.mark.parametrize("T", [50, 1300])
def test_backward_strides(T):
    c = Case(T, 128, 97, 16, 2)
    _, h = M.lora_add(c.y, c.x, c.adapters, c.ids, save_for_backward=True)
    want = M.lora_add_backward(c.dy, c.x, h, c.adapters, c.ids)
    for left, pitch in ((0, 104), (8, 112), (3, 101)):
        dy = torch.full((T, pitch), float("nan"), dtype=BF16, device="cuda")
        dy[:, left:left + 97] = c.dy
        x = torch.full((T, 144), float("nan"), dtype=BF16, device="cuda")
        x[:, :128] = c.x
        dx = torch.full((T, 131 + left), 7.0, dtype=BF16, device="cuda")
        dx[:, left:left + 128] = 0
        got = M.lora_add_backward(dy[:, left:left + 97], x[:, :128], h, c.adapters, c.ids, dx=dx[:, left:left + 128])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (dx[:, :left] == 7).all() and (dx[:, left + 128:] == 7).all()


# The same of tiles of 128 rows, which take over where there are many rows (few_rows in csrc/lora.cu: for small K and N late).
@pytest.mark.parametrize("body", [
    lambda T: test_without_scales_and_in_place(T), lambda T: test_one_adapter_or_none(T, "none"), lambda T: test_one_adapter_or_none(T, "last"),
    lambda T: test_strides_and_alignment(T), lambda T: test_bad_ids_are_reported(T), lambda T: test_nonfinite_rows_stay_theirs(T),
    lambda T: test_fp16_h_of_any_size(T, 2.0 ** -18), lambda T: test_fp16_h_of_any_size(T, 2.0 ** 6),
    lambda T: test_backward_of_one_adapter_or_none(T, "none"), lambda T: test_backward_of_one_adapter_or_none(T, "one"),
    lambda T: test_backward_of_one_adapter_or_none(T, "sorted"), lambda T: test_backward_bad_ids(T), lambda T: test_backward_strides(T)])
def test_in_tiles_of_128(body):
    body(40000)


@pytest.mark.parametrize("shape", [(60000, 8, 1, 128, 1), (60001, 16, 3, 128, 5), (40000, 128, 64, 64, 1000)])
def test_many_rows_of_small_sizes(shape):
    check(Case(*shape))
    check_backward(Case(*shape))
    assert M.nvfp4_get_device_error() == 0


def test_gradients_on_any_boundary():
    c = Case(300, 264, 40, 16, 3)
    _, h = M.lora_add(c.y, c.x, c.adapters, c.ids, save_for_backward=True)
    want = M.lora_add_backward(c.dy, c.x, h, c.adapters, c.ids)
    a, ws = c.adapters, torch.empty(M.lib().lora_add_backward_workspace_bytes(300, 3, 16, 264, 40), dtype=torch.uint8, device="cuda")
    down, up = (torch.full((t.numel() + 2,), 7.0, device="cuda") for t in want[1:])
    dx = torch.empty_like(want[0])
    assert M.lib().lora_add_backward(a.struct, c.dy.data_ptr(), 40, c.x.data_ptr(), 264, h.data_ptr(), c.ids.data_ptr(), 300,
                                     dx.data_ptr(), 264, 1, 0, down.data_ptr() + 4, up.data_ptr() + 4, ws.data_ptr(), ws.numel(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dx, want[0])
    for got, w in ((down, want[1]), (up, want[2])):
        assert torch.equal(got[1:-1], w.flatten()) and got[0] == 7 and got[-1] == 7
