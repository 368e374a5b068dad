"""lora_add and its gradient where offsets pass 32 bits, and gradients beside rows with NaN and infinities."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
PITCH = 1 << 22                            # 600 rows of it: 5 GB of 16-bit elements


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    M.lib()
    M.nvfp4_get_device_error()
    yield
    torch.cuda.empty_cache()


def draw(seed, dtype, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


def apart(t, pitch):
    """The same rows, `pitch` elements apart."""
    rows = torch.empty((t.shape[0] - 1) * pitch + t.shape[1], dtype=t.dtype, device="cuda").as_strided(t.shape, (pitch, 1))
    return rows.copy_(t)


# Tiles of 128 rows; rows of y, out, dy and dx on 16-byte boundaries, and on none (an odd pitch).
@pytest.mark.parametrize("odd", [0, 1])
def test_rows_past_32_bits_in_tiles_of_128(odd):
    T, K, N, R, L = 600, 2048, 2048 - odd, 64, 2
    adapters = M.LoRAAdapters(draw(1, BF16, L, R, K) / 32, draw(2, BF16, L, N, R))
    x, y, dy = draw(3, BF16, T, K), draw(4, BF16, T, N), draw(5, BF16, T, N)
    ids = torch.arange(T, device="cuda").remainder(3).sub(1).to(torch.int32)
    want, h = M.lora_add(y, x, adapters, ids, save_for_backward=True)
    grads = M.lora_add_backward(dy, x, h, adapters, ids)
    far_x, far_y = apart(x, PITCH), apart(y, PITCH + odd)
    got, got_h = M.lora_add(far_y, far_x, adapters, ids, save_for_backward=True)
    assert torch.equal(got, want) and torch.equal(got_h, h)
    assert torch.equal(M.lora_add(far_y, far_x, adapters, ids, out=far_y), want)
    far_y.copy_(dy)
    dx = apart(torch.zeros(T, K, dtype=BF16, device="cuda"), PITCH + odd)
    got = M.lora_add_backward(far_y, far_x, h, adapters, ids, dx=dx)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert M.nvfp4_get_device_error() == 0


# 2^32 elements of A, or of B, in tiles of 16 rows and of 128; the last adapter's lie behind 2^31.
@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("K,N", [(1 << 18, 64), (64, 1 << 18)])
def test_adapters_past_32_bits(T, K, N):
    L, R, used = 256, 64, [0, 3, 255]
    down, up = draw(1, BF16, 3, R, K) / K ** 0.5, draw(2, BF16, 3, N, R)
    few, which = M.LoRAAdapters(down, up), torch.arange(T, device="cuda").remainder(3)
    x, y, dy = draw(3, BF16, T, K), draw(4, BF16, T, N), draw(5, BF16, T, N)
    few_ids = which.to(torch.int32)
    want, h = M.lora_add(y, x, few, few_ids, save_for_backward=True)
    want_grads = M.lora_add_backward(dy, x, h, few, few_ids)
    all_down, all_up = torch.zeros(L, R, K, dtype=BF16, device="cuda"), torch.zeros(L, N, R, dtype=BF16, device="cuda")
    all_down[used], all_up[used] = down, up
    many, ids = M.LoRAAdapters(all_down, all_up), torch.tensor(used, device="cuda")[which].to(torch.int32)
    got, got_h = M.lora_add(y, x, many, ids, save_for_backward=True)
    assert torch.equal(got, want) and torch.equal(got_h, h)
    dx, ddown, dup = M.lora_add_backward(dy, x, h, many, ids)
    assert torch.equal(dx, want_grads[0])
    for grad, w in ((ddown, want_grads[1]), (dup, want_grads[2])):
        # sums of the same products, cut into other parts: T <= 600 terms, added in FP32 and on the tensor cores (2^-22 a step)
        assert torch.linalg.vector_norm((grad[used] - w).double()) <= 2.0 ** -17 * torch.linalg.vector_norm(w.double())
        for a in (1, 2, 100, 254):
            assert not grad[a].any()
    assert M.nvfp4_get_device_error() == 0


@pytest.mark.parametrize("T,K,N,R", [(50, 128, 97, 16), (1300, 264, 200, 40), (2000, 1024, 1024, 64), (9000, 512, 1031, 16)])
@pytest.mark.parametrize("last", [False, True])
def test_gradients_of_other_adapters_beside_nonfinite_rows(T, K, N, R, last):
    L = 5
    adapters = M.LoRAAdapters(draw(1, BF16, L, R, K) / 16, draw(2, BF16, L, N, R))
    x, dy = draw(3, BF16, T, K), draw(4, BF16, T, N)
    ids = torch.arange(T, device="cuda").remainder(L + 1).sub(1).to(torch.int32)
    of = lambda a: int((ids == a).nonzero().flatten()[-1 if last else 2])  # noqa: E731
    h = M.lora_add(dy, x, adapters, ids, save_for_backward=True)[1]
    want = M.lora_add_backward(dy, x, h, adapters, ids)
    x[of(0), 5], dy[of(1), 2], x[of(-1), 1], dy[of(-1), 1] = (float(v) for v in ("nan", "inf", "nan", "nan"))
    dx, ddown, dup = M.lora_add_backward(dy, x, h, adapters, ids)
    # x's NaN is in a column of its adapter's dA; dy's infinity in its row of dx, its adapter's dA and a row of its dB
    rows = torch.arange(T, device="cuda") != of(1)
    assert torch.equal(dx[rows], want[0][rows]) and not dx[of(1)].isfinite().any()
    columns = torch.arange(K, device="cuda") != 5
    assert ddown[0, :, 5].isnan().all() and torch.equal(ddown[0][:, columns], want[1][0][:, columns])
    assert not ddown[1].isfinite().any() and torch.equal(ddown[2:], want[1][2:])
    outputs = torch.arange(N, device="cuda") != 2
    assert not dup[1, 2].isfinite().any() and torch.equal(dup[1][outputs], want[2][1][outputs])
    assert torch.equal(dup[0], want[2][0]) and torch.equal(dup[2:], want[2][2:])
    assert M.nvfp4_get_device_error() == 0
