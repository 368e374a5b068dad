"""lora_add and dx with long rows, against 64 bits: how far the sums over K (over N in dx) are off does not grow with the chains.

Tolerances.  All values are of one sign, so a sum's terms add up to it.  A chain of at most 32 m16n8k16 steps, each off by at most
2^-22 of the accumulator; 8 sub-slices to a group for every 32768 columns, in FP32 one after the other, and three joins of groups (2^-24
each).  dx in FP32: dh as three BF16 terms leaves 2^-24, its products (3 R / 16 + 4) 2^-22, the sum one rounding; the scale another."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LENGTHS = [8, 1032, 32768, 32776, 70000, 262144, 1 << 20]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()


def draw(seed, dtype, *shape):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.rand(*shape, device="cuda", generator=g).to(dtype)


def product(a, b):
    """a b^T in 64 bits, the columns in pieces."""
    return sum(a[:, c:c + 65536].double() @ b[:, c:c + 65536].double().T for c in range(0, a.shape[1], 65536))


def sum_bound(columns):
    return 32 * 2.0 ** -22 + (8 * ((columns + 32767) // 32768) + 3) * 2.0 ** -24


@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("R,dtype,out", [(8, BF16, BF16), (64, BF16, F32), (24, F16, F16), (128, BF16, BF16)])
def test_long_rows(K, R, dtype, out):
    T, N = 600, 64
    x, down, up = draw(K, dtype, T, K), (draw(R, dtype, 1, R, K).float() / K).to(BF16).to(dtype), draw(3, dtype, 1, N, R)
    down.clamp_(min=2.0 ** -24)                                   # FP16 has no smaller steps
    adapters, y = M.LoRAAdapters(down, up), torch.zeros(T, N, dtype=out, device="cuda")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    got, h = M.lora_add(y, x, adapters, ids, save_for_backward=True)
    want = product(x, down[0])
    assert ((h.double() - want).abs() <= sum_bound(K) * want).all()
    for at in (slice(0, 1), slice(100, 117), slice(300, 556)):    # a row does not depend on the others
        one, one_h = M.lora_add(y[at], x[at], adapters, ids[at], save_for_backward=True)
        assert torch.equal(one, got[at]) and torch.equal(one_h, h[at])
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("N", LENGTHS + [100001])
@pytest.mark.parametrize("R", [8, 64])
def test_long_rows_of_dy(N, R):
    T, K = 600, 72
    x, dy, down = draw(1, BF16, T, K), draw(2, BF16, T, N), draw(4, BF16, 1, R, K)
    up = (draw(3, F32, 1, N, R) / N).to(BF16)
    adapters, ids = M.LoRAAdapters(down, up, torch.full((1,), 0.7, device="cuda")), torch.zeros(T, dtype=torch.int32, device="cuda")
    h = draw(5, F32, T, R)
    dx = M.lora_add_backward(dy, x, h, adapters, ids, dx=torch.zeros(T, K, device="cuda"))[0]
    want = product(product(dy, up[0].T) * adapters.tensors[2].double(), down[0].double().T)
    assert ((dx.double() - want).abs() <= 1.01 * (sum_bound(N) + 3 * 2.0 ** -24 + (3 * R / 16 + 4) * 2.0 ** -22) * want).all()
    for at in (slice(0, 1), slice(100, 117)):
        one = M.lora_add_backward(dy[at], x[at], h[at], adapters, ids[at], dx=torch.zeros(at.stop - at.start, K, device="cuda"))[0]
        assert torch.equal(one, dx[at])
    assert M.nvfp4_get_device_error() == 0
