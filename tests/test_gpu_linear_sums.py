"""Dense 4-bit products of operands of one sign, whose sums grow with every step.

Bound.  A product of 64 K-elements is added to the FP32 accumulator in one step, K / 64 of them; the tensor cores may
drop what lies below the accumulator's last place, 2^-23 of the running sum, and the sum within a step as much again;
the outer scales, the bias and the output are four roundings of 2^-24.  With no sign changes the running sum is at most
the result: |error| <= (2 K / 64 + 2) 2^-23 sum_k x_k w_k.  (Measured: 30 units of 2^-24 at K = 8192 NVFP4, which is
more than the 2^-20 that operands of mixed signs stay within.)"""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import mxfp4 as X
from oracle import quant as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T,N", [(2, 150), (40, 150), (2400, 2100)])     # each of the kernels
@pytest.mark.parametrize("K", [64, 2048, 8192])
def test_operands_of_one_sign(mx, T, N, K):
    g = torch.Generator().manual_seed(K + T)
    # blocks of different magnitudes, so that the scales take part
    x = (torch.rand(T, K, generator=g) * torch.exp2(torch.randint(-4, 5, (T, 1), generator=g).float())).to(torch.bfloat16)
    w = (torch.rand(N, K, generator=g) * torch.exp2(torch.randint(-3, 4, (1, K // 32), generator=g).float())
         .repeat_interleave(32, 1)).to(torch.bfloat16)
    rows = torch.arange(0, T, max(1, T // 100))
    cols = torch.arange(0, N, max(1, N // 200))
    quantise = (lambda a: X.dequantize_rows(*X.quantize_rows(a))) if mx else (lambda a: Q.dequantize_rows(*Q.quantize_rows(a)))
    want = quantise(x[rows].float().numpy()) @ quantise(w[cols].float().numpy()).T
    linear, wq = (M.mxfp4_linear, M.mxfp4_quantize_weight) if mx else (M.nvfp4_linear, M.nvfp4_quantize_weight)
    y = linear(x.cuda(), wq(w.cuda()), out_dtype=torch.float32).cpu()[rows][:, cols].double().numpy()
    assert np.all(np.abs(y - want) <= (2 * K / 64 + 2) * 2.0 ** -23 * want)
    assert M.nvfp4_get_device_error() == 0
