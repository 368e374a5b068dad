"""A row of x with an Inf or NaN gives a row of NaN from either dense product, in each of its kernels, whatever the
weights, the bias and the output's type are; the other rows keep their bits and the device error says so."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T,N,K", [(1, 64, 64), (9, 96, 256), (16, 77, 2048), (40, 96, 256), (300, 500, 8192), (2400, 2100, 256),
                                   (2400, 2101, 256)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_non_finite_rows_give_nan(mx, T, N, K, bad):
    g = torch.Generator("cuda").manual_seed(T + N)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randn(N, K, device="cuda", generator=g).to(torch.bfloat16)
    w[3] = 0                                                 # an output with no weights
    bias = torch.randn(N, device="cuda", generator=g)
    linear, wq = (M.mxfp4_linear, M.mxfp4_quantize_weight(w)) if mx else (M.nvfp4_linear, M.nvfp4_quantize_weight(w))
    rows = sorted({T - 1, T // 3})
    broken = x.clone()
    for i, t in enumerate(rows):
        broken[t, (5 + 31 * i) % K] = bad
    for out_dtype in (torch.float32, torch.bfloat16, torch.float16):
        want = linear(x, wq, bias=bias, out_dtype=out_dtype)
        assert M.nvfp4_get_device_error() == 0
        got = linear(broken, wq, bias=bias, out_dtype=out_dtype)
        assert M.nvfp4_get_device_error() == 6               # NVFP4_ERR_NONFINITE
        assert bool(torch.isnan(got[rows]).all())
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[rows] = False
        assert torch.equal(got[keep], want[keep])
