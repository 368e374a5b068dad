"""GPU parity of mxfp4_linear and nvfp4_linear.

The operands are quantised by the oracle from the same values (bit-equal to the library's rows),
their products are summed exactly in FP64, and the tensor cores' FP32 accumulation is held to
|error| <= 2^-20 sum_k |x_k w_k| per element (K / 64 <= 128 additions of at most 2^-24 of the running
sum, and the scaling's three roundings) and to a relative L2 of 1e-5; a 16-bit output may differ from the
exact value by that and by half a unit in its last place.
"""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import mxfp4 as X
from oracle import quant as Q
from _helpers import GEMM_REL_L2

pytestmark = pytest.mark.gpu
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def rows64(x, mx):
    x = x.float().cpu().numpy()
    return X.dequantize_rows(*X.quantize_rows(x)) if mx else Q.dequantize_rows(*Q.quantize_rows(x))


def make(T, N, K, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * T + 5 * N + K)
    x = torch.randn(T, K, generator=g) * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g).float())
    w = 0.05 * torch.randn(N, K, generator=g)
    return x.to(dtype).cuda(), w.to(torch.bfloat16).cuda()


def weight(w, mx):
    return M.mxfp4_quantize_weight(w) if mx else M.nvfp4_quantize_weight(w)


def linear(mx):
    return M.mxfp4_linear if mx else M.nvfp4_linear


def check(x, w, mx, out_dtype=torch.float32, bias=None):
    y = linear(mx)(x, weight(w, mx), bias=bias, out_dtype=out_dtype)
    assert y.dtype == out_dtype and tuple(y.shape) == (x.shape[0], w.shape[0])
    a, b = rows64(x, mx), rows64(w, mx)
    want = a @ b.T
    if bias is not None:
        want = want + bias.double().cpu().numpy()[None, :]
    size = np.abs(a) @ np.abs(b).T + (0 if bias is None else np.abs(bias.double().cpu().numpy())[None, :])
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -20 * size + UNIT[out_dtype] * np.abs(want) + 1e-30), (err / (size + 1e-30)).max()
    if out_dtype == torch.float32:
        assert np.linalg.norm(err) <= GEMM_REL_L2 * max(np.linalg.norm(want), 1e-30)
    assert M.nvfp4_get_device_error() == 0
    return y


@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 128, 64), (2, 31, 96), (16, 64, 128), (17, 33, 160), (31, 257, 288),
                                   (128, 256, 256), (129, 100, 512), (130, 1000, 320), (300, 520, 1056), (1, 5000, 2048),
                                   (64, 2000, 4096), (700, 4100, 256), (2500, 2100, 192), (40, 9, 16384),
                                   # few tokens, several tiles to an SM and more stages than fit; the same for many
                                   (3, 33000, 544), (1, 12000, 8192), (2, 300, 8160), (16, 20000, 96), (4, 100, 8192),
                                   (200, 20000, 288), (1000, 8200, 352), (3000, 5000, 1056)])
def test_mxfp4_shapes(T, N, K):
    check(*make(T, N, K), True)


@pytest.mark.parametrize("T,N,K", [(1, 1, 64), (1, 128, 128), (2, 31, 192), (16, 64, 256), (17, 33, 320), (31, 257, 448),
                                   (129, 100, 512), (130, 1000, 320), (300, 520, 1088), (1, 5000, 2048), (64, 2000, 4096),
                                   (700, 4100, 256), (2500, 2100, 192), (40, 9, 8192),
                                   (3, 33000, 576), (1, 12000, 8192), (2, 300, 8128), (16, 20000, 128), (4, 100, 8192),
                                   (200, 20000, 320), (1000, 8200, 320), (3000, 5000, 1088), (50, 70, 3136), (33, 64, 6080)])
def test_nvfp4_shapes(T, N, K):
    check(*make(T, N, K), False)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [64, 77, 300])
def test_output_types_and_bias(mx, out_dtype, N):
    x, w = make(150, N, 256)
    bias = torch.randn(N, device="cuda", generator=torch.Generator("cuda").manual_seed(N))
    check(x, w, mx, out_dtype, bias)
    check(x, w, mx, out_dtype)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [2104, 2101, 2052])              # rows on 16-byte boundaries or not, ends inside a tile
def test_output_types_of_many_tokens(mx, out_dtype, N):
    x, w = make(2350, N, 320)
    check(x, w, mx, out_dtype, torch.randn(N, device="cuda", generator=torch.Generator("cuda").manual_seed(N)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 9, 33])
@pytest.mark.parametrize("offset,pitch", [(0, 2080), (8, 2104), (4, 2084), (3, 2085)])   # 32-, 16- and 8-byte aligned rows, odd ones
def test_mxfp4_input_types(dtype, T, offset, pitch):
    x, w = make(T, 200, 2080, dtype)
    wide = torch.zeros((T, pitch + offset), dtype=dtype, device="cuda")
    wide[:, offset:offset + 2080] = x
    check(wide[:, offset:offset + 2080], w, True)


@pytest.mark.parametrize("mx", [True, False])
def test_zero_rows_and_channels(mx):
    x, w = make(40, 96, 256)
    x[3] = 0
    x[:, 64:128] = 0
    w[5] = 0
    y = check(x, w, mx)
    assert not bool(y[3].any()) and not bool(y[:, 5].any())


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T,N", [(9, 96), (40, 96), (2400, 2100)])      # each of the kernels
def test_a_non_finite_row_stays_its_own(mx, T, N):
    x, w = make(T, N, 256)
    want = linear(mx)(x, weight(w, mx))
    x[7, 100] = float("inf")
    got = linear(mx)(x, weight(w, mx))
    assert M.nvfp4_get_device_error() == 6
    keep = [t for t in range(T) if t != 7]
    assert torch.equal(got[keep], want[keep])
    if mx:
        assert bool(torch.isnan(got[7]).all())


@pytest.mark.parametrize("mx", [True, False])
def test_batch_invariance(mx):
    # every tile width and row count takes K in the same order: the same bits
    x, w = make(2300, 1100, 1024)
    wq = weight(w, mx)
    full = linear(mx)(x, wq, out_dtype=torch.float32)
    for lo, hi in ((0, 1), (5, 6), (0, 16), (3, 20), (100, 133), (0, 128), (64, 321), (0, 1000), (1000, 2300)):
        assert torch.equal(linear(mx)(x[lo:hi], wq, out_dtype=torch.float32), full[lo:hi]), (lo, hi)
    # nor does an output's value depend on which other outputs there are
    part = weight(w[128:200].contiguous(), mx)
    assert torch.equal(linear(mx)(x, part, out_dtype=torch.float32), full[:, 128:200])


@pytest.mark.parametrize("mx", [True, False])
def test_strides_and_given_output(mx):
    x, w = make(60, 136, 256)
    wq = weight(w, mx)
    want = linear(mx)(x, wq)
    wide = torch.zeros((60, 600), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264] = x
    assert torch.equal(linear(mx)(wide[:, 8:264], wq), want)
    twice = x.repeat_interleave(2, 0)
    assert torch.equal(linear(mx)(twice[::2], wq), want)
    if mx:
        odd = torch.zeros((60, 301), dtype=torch.bfloat16, device="cuda")
        odd[:, 3:259] = x
        assert torch.equal(M.mxfp4_linear(odd[:, 3:259], wq), want)
    for lo, n in ((0, 200), (5, 201), (8, 160)):
        out = torch.full((60, n), 7.0, dtype=torch.bfloat16, device="cuda")
        got = linear(mx)(x, wq, out=out[:, lo:lo + 136])
        assert torch.equal(got, want)
        rest = torch.ones(n, dtype=torch.bool)
        rest[lo:lo + 136] = False
        assert bool((out[:, rest.cuda()] == 7.0).all())
    assert linear(mx)(x[:0], wq).shape == (0, 136)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N", [(5, 95), (40, 95), (300, 77), (2350, 2051)])          # each of the kernels
def test_output_rows_on_every_boundary(mx, out_dtype, T, N):
    x, w = make(T, N, 256)
    wq = weight(w, mx)
    bias = torch.randn(N, device="cuda", generator=torch.Generator("cuda").manual_seed(N))
    want = linear(mx)(x, wq, bias=bias, out_dtype=out_dtype)
    # row pitches and starts of an odd number of elements, of two, of four, of eight and sixteen
    for lo, pitch in ((0, N + 4 - N % 4), (1, N + 2), (2, N + 4 - N % 2), (3, N + 9), (4, N + 24 - N % 8), (16, N + 48 - N % 16)):
        out = torch.full((T, pitch), 7.0, dtype=out_dtype, device="cuda")
        assert torch.equal(linear(mx)(x, wq, bias=bias, out=out[:, lo:lo + N]), want)
        rest = torch.ones(pitch, dtype=torch.bool, device="cuda")
        rest[lo:lo + N] = False
        assert bool((out[:, rest] == 7.0).all())


@pytest.mark.parametrize("mx", [True, False])
def test_refusals(mx):
    x, w = make(4, 32, 128)
    wq = weight(w, mx)
    f = linear(mx)
    with pytest.raises(ValueError):
        f(x[:, :64], wq)
    with pytest.raises(ValueError):
        f(x, weight(w, not mx))
    with pytest.raises(ValueError):
        f(x, wq, bias=torch.zeros(31, device="cuda"))
    with pytest.raises(ValueError):
        f(x, wq, out=torch.zeros((4, 33), device="cuda"))
    with pytest.raises(ValueError):
        f(x, wq, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        f(x.t().contiguous().t(), wq)
    if not mx:
        with pytest.raises(ValueError):
            f(x.float(), wq)
    if mx:
        y = M.mxfp4_linear(x, M.mxfp4_weight_from_codes(wq.tensors[0][:32], torch.full((32, 4), 127, dtype=torch.uint8,
                                                                                       device="cuda")))
        assert y.shape == (4, 32)


@pytest.mark.parametrize("mx", [True, False])
def test_another_stream_and_graph(mx):
    x, w = make(200, 300, 512)
    wq = weight(w, mx)
    want = linear(mx)(x, wq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [linear(mx)(x, wq, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(g):
        linear(mx)(x, wq, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("mx", [True, False])
def test_offsets_past_32_bits(mx):
    # outputs past element 2^31
    T, N, K = 70000, 32000, 64
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randn(N, K, device="cuda", generator=g).to(torch.bfloat16)
    wq = weight(w, mx)
    y = linear(mx)(x, wq)
    assert torch.equal(y[-200:], linear(mx)(x[-200:], wq))
    assert torch.equal(y[:200], linear(mx)(x[:200], wq))
    assert M.nvfp4_get_device_error() == 0
