"""The balance loss with masks of either type, and with rows past 32 bits."""

import numpy as np
import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B
from oracle import balance as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()
    yield
    torch.cuda.empty_cache()


def make(T, E, k, dtype):
    g = torch.Generator("cuda").manual_seed(T + E)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return n(T, E).to(dtype), n(T, E).topk(k).indices.to(torch.int32), n(T) > -0.5


def both(logits, ids, **kw):
    b = M.moe_balance_loss(logits, ids, **kw)
    dloss = torch.ones_like(b.loss)
    back = lambda **more: M.moe_balance_loss_backward(logits, ids.shape[1], b.counts, b.tokens, dloss, **kw, **more)  # noqa: E731
    return [*b, back(), back(dlogits=torch.ones(logits.shape, dtype=logits.dtype, device="cuda"))]


@pytest.mark.parametrize("T,E", [(40, 128), (9000, 60)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_mask_of_bytes(T, E, score):
    logits, ids, mask = make(T, E, 4, torch.bfloat16)
    cut = torch.tensor([0, T // 3, T - 3], dtype=torch.int32, device="cuda")
    want = both(logits, ids, score=score, mask=mask, seq_offsets=cut)
    ones = mask.to(torch.uint8)
    for bytes_ in (ones, ones * 255, ones * torch.randint(1, 256, (T,), device="cuda").to(torch.uint8)):
        assert all(torch.equal(a, b) for a, b in zip(both(logits, ids, score=score, mask=bytes_, seq_offsets=cut), want))
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("dtype,pitch", [(torch.float32, 1 << 22), (torch.bfloat16, (1 << 22) + 1)])
@pytest.mark.parametrize("E", [128, 1000])
def test_rows_past_32_bits(dtype, pitch, E):
    T = 600                                                       # one kernel with 128 experts, two with 1000
    logits, ids, mask = make(T, E, 4, dtype)
    want = both(logits, ids, mask=mask)
    far = torch.empty((T - 1) * pitch + E, dtype=dtype, device="cuda").as_strided((T, E), (pitch, 1)).copy_(logits)
    got = M.moe_balance_loss(far, ids, mask=mask)
    # by the width of the loads a lane has other experts, and sums come in another order: two sums of T terms
    assert torch.equal(got.counts, want[1]) and torch.equal(got.tokens, want[3])
    assert torch.allclose(got.probs, want[2], rtol=2e-5, atol=0) and torch.allclose(got.loss, want[0], rtol=2e-5, atol=0)
    out = torch.empty((T - 1) * pitch + E, dtype=dtype, device="cuda").as_strided((T, E), (pitch, 1)).copy_(torch.zeros_like(logits))
    grad = M.moe_balance_loss_backward(far, 4, got.counts, got.tokens, torch.ones(1, device="cuda"), mask=mask, dlogits=out)
    exact, size = O.backward(logits.cpu().double().numpy(), 4, got.counts.cpu().numpy(), got.tokens.cpu().numpy(), [1.0], "softmax",
                             mask.cpu().numpy())
    off = np.abs(grad.cpu().double().numpy() - exact)             # test_gpu_balance.py derives the bound
    assert np.all(off <= 2e-5 * size + torch.finfo(dtype).eps / 2 * np.abs(exact) + 1e-38)
    assert not grad[~mask].any() and M.nvfp4_get_device_error() == 0
