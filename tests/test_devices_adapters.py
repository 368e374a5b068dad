"""Tensors that are not on the current device are refused by the balance loss and the adapters before anything is launched."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from test_devices import Tensor, bf16, device_0, f32, i32  # noqa: F401


def adapters():
    return M.LoRAAdapters(Tensor(bf16, 2, 16, 64), Tensor(bf16, 2, 40, 16))


@pytest.mark.parametrize("call", [
    lambda: M.moe_balance_loss(Tensor(f32, 8, 64), Tensor(i32, 8, 4)),
    lambda: M.moe_balance_loss_backward(Tensor(f32, 8, 64), 4, Tensor(i32, 1, 64), Tensor(i32, 1), Tensor(f32, 1)),
    lambda: M.lora_add(Tensor(bf16, 8, 40), Tensor(bf16, 8, 64), adapters(), Tensor(i32, 8)),
    lambda: M.lora_add_backward(Tensor(bf16, 8, 40), Tensor(bf16, 8, 64), Tensor(f32, 8, 16), adapters(), Tensor(i32, 8)),
], ids=["balance_loss", "balance_loss_backward", "lora_add", "lora_add_backward"])
def test_tensors_of_another_device(call, device_0):  # noqa: F811
    with pytest.raises(ValueError, match="current device"):
        call()


def test_adapters_elsewhere():
    a = adapters()
    x = torch.zeros(4, 64, dtype=bf16)
    assert a.device == torch.device("cuda", 1) and (a.L, a.R, a.K, a.N) == (2, 16, 64, 40)
    with pytest.raises(ValueError):
        M.lora_add(x[:, :40], x, a, torch.zeros(4, dtype=i32))
