"""GPU parity of the MXFP4 row quantiser and its inverse against oracle/mxfp4.py: every step is
exact but one rounding that both take the same way, so codes, scales and values are bit-equal."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import mxfp4 as X
from oracle import quant as Q

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def check(x):
    rows, cols = x.shape
    codes, sf = M.mxfp4_quantize_rows(x)
    want_c, want_s = X.quantize_rows(x.float().cpu().numpy())
    got = codes.cpu().numpy()
    assert np.array_equal(got[:rows], Q.pack_nibbles(want_c)) and not got[rows:].any()
    tiles = sf.cpu().numpy()
    index = X.sf_byte_index(rows, cols)
    assert np.array_equal(tiles[index], want_s)
    rest = np.ones(tiles.size, bool)
    rest[index.ravel()] = False
    assert not tiles[rest].any()                              # pad rows and pad blocks
    want_v = X.dequantize_rows(want_c, want_s)
    for dtype in (torch.bfloat16, torch.float32):
        v = M.mxfp4_dequantize_rows(codes, sf, rows, cols, dtype=dtype)
        assert v.dtype == dtype and np.array_equal(v.double().cpu().numpy(), want_v, equal_nan=True)
    return want_c, want_s


def make(rows, cols, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g).float())
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (128, 96), (129, 128), (33, 160), (5, 2080), (257, 4096),
                                       (2, 16384), (1, 1 << 20)])
def test_shapes(dtype, rows, cols):
    check(make(rows, cols, dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_values_at_the_edges(dtype):
    f = torch.finfo(dtype)
    x = torch.zeros((8, 64), dtype=dtype)
    x[0, :4] = torch.tensor([f.max, -f.max, f.tiny, -f.tiny], dtype=dtype)
    x[1, :3] = torch.tensor([f.smallest_normal, -f.smallest_normal / 2, f.smallest_normal / 4], dtype=dtype)
    x[2, 0] = f.smallest_normal * f.eps                        # the smallest subnormal alone
    x[3] = -0.0
    x[4, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, -0.25, -0.75, -5.0, -7.5, 0.1, 4.0],
                             dtype=dtype)                      # ties and saturation at scale 1
    x[5, 32:] = 3.0
    x[6] = torch.linspace(-6, 6, 64).to(dtype)
    check(x.cuda())
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_non_finite_blocks(dtype, bad):
    x = make(4, 128, dtype)
    x[2, 70] = bad
    codes, scales = check(x)
    assert scales[2].tolist().count(255) == 1 and M.nvfp4_get_device_error() == 6


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_alignment(dtype):
    big = make(40, 300, dtype)
    for view in (big[:, :256], big[:, 1:65], big[::3, 8:168], big[:, 3:35]):
        a, b = M.mxfp4_quantize_rows(view), M.mxfp4_quantize_rows(view.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    codes, sf = M.mxfp4_quantize_rows(big[:0, :64])
    assert codes.numel() == 0 and M.mxfp4_dequantize_rows(codes, sf, 0, 64).shape == (0, 64)


def test_weight_from_codes():
    x = make(70, 416, torch.bfloat16)
    c, s = X.quantize_rows(x.float().cpu().numpy())
    w = M.mxfp4_weight_from_codes(torch.from_numpy(Q.pack_nibbles(c)).cuda(), torch.from_numpy(s).cuda())
    codes, sf = M.mxfp4_quantize_rows(x)
    assert (w.N, w.K) == (70, 416) and torch.equal(w.tensors[0], codes) and torch.equal(w.tensors[1], sf)


def test_another_stream():
    x = make(600, 1024, torch.bfloat16)
    want = M.mxfp4_quantize_rows(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.mxfp4_quantize_rows(x, stream=s)
    v = M.mxfp4_dequantize_rows(*got, 600, 1024, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(v, M.mxfp4_dequantize_rows(*want, 600, 1024))


def test_offsets_past_32_bits():
    rows, cols = 262144 + 3, 8192                              # 2^31 elements and three rows more
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = make(3, cols, torch.bfloat16)
    x[-3:] = tail
    codes, sf = M.mxfp4_quantize_rows(x)
    v = M.mxfp4_dequantize_rows(codes, sf, rows, cols)
    want = M.mxfp4_dequantize_rows(*M.mxfp4_quantize_rows(tail), 3, cols)
    assert torch.equal(v[-3:], want) and not bool(v[:-3].any())
