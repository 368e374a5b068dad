"""lora_add and lora_add_backward with more tiles of 128 rows than clusters run at once: a cluster's tiles follow one another, and
a row has the bits that it has in a batch of few rows (tiles of 16, whose values the oracle's tests check)."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def make(T, K, N, R, L, dtype, out):
    g = torch.Generator("cuda").manual_seed(T + K + N + R)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    adapters = M.LoRAAdapters((n(L, R, K) / K ** 0.5).to(dtype), (0.1 * n(L, N, R)).to(dtype), 0.5 + n(L).abs())
    return n(T, K).to(dtype), n(T, N).to(out), adapters, torch.randint(-1, L, (T,), device="cuda", generator=g).to(torch.int32)


# A CTA's share of the columns that the first product sums (K, and N in dx) ends after five stages of 64: 257 to 320 columns of
# the first CTA, 769 to 832 of the second; 384 and 1024 beside them.
@pytest.mark.parametrize("columns", [264, 320, 384, 800, 832, 1024])
@pytest.mark.parametrize("other,R,L,out", [(4096, 64, 1, BF16), (520, 64, 300, BF16), (2048, 48, 3, F32), (1000, 40, 40, F16)])
def test_many_tiles_to_a_cluster(columns, other, R, L, out):
    T = 20000
    some = [torch.randperm(T, generator=torch.Generator().manual_seed(i))[:250].cuda() for i in range(8)]
    x, y, adapters, ids = make(T, columns, other, R, L, BF16, out)
    for _ in range(3):
        got, h = M.lora_add(y, x, adapters, ids, save_for_backward=True)
        for at in some:
            one, one_h = M.lora_add(y[at], x[at], adapters, ids[at], save_for_backward=True)
            assert torch.equal(got[at], one) and torch.equal(h[at], one_h)
    x, dy, adapters, ids = make(T, other // 8 * 8, columns, R, L, BF16, BF16)
    h = torch.randn(T, R, device="cuda", generator=torch.Generator("cuda").manual_seed(R))
    base = torch.zeros(T, x.shape[1], dtype=out, device="cuda")
    first = None
    for _ in range(3):
        grads = M.lora_add_backward(dy, x, h, adapters, ids, dx=base.clone())
        for at in some:
            assert torch.equal(grads[0][at], M.lora_add_backward(dy[at], x[at], h[at], adapters, ids[at], dx=base[at])[0])
        first = first or grads
        assert all(torch.equal(a, b) for a, b in zip(grads, first))
    assert M.nvfp4_get_device_error() == 0
