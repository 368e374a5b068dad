"""Tensors and streams that do not belong to the current device are refused before anything is
launched: the library launches on the current device, where such memory cannot be used."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M
from nvfp4_moe_expert_gb300 import build as B


class Tensor:
    """What the binding looks at of a CUDA tensor on device 1 (no such device is needed)."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)
        self.device = torch.device("cuda", 1)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        strides = torch.empty(self.shape, device="meta").stride()
        return strides if i is None else strides[i]

    def contiguous(self):
        return self

    def is_contiguous(self):
        return True

    def get_device(self):
        return 1

    def data_ptr(self):
        return 1 << 20


class Stream:
    cuda_stream = 0

    def __init__(self, device_index):
        self.device_index = device_index


@pytest.fixture(autouse=True)
def device_0(monkeypatch):
    """Device 0 is the current one, and a call that gets as far as the library fails the test."""
    B.build()
    M.lib()
    monkeypatch.setattr(M, "_current_device", lambda: 0)

    class Library:
        def __getattr__(self, name):
            if name in ("nvfp4_rows_padded", "nvfp4_sf_bytes", "moe_workspace_layout_query"):
                return getattr(real, name)
            raise AssertionError(f"{name} was reached")

    real = M.lib()
    monkeypatch.setattr(M, "lib", lambda: Library())


f32, bf16, i32, u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def weights():
    return M.MoEWeights(*[Tensor(u8, 8)] * 6, 4, 256, 128)


@pytest.mark.parametrize("call", [
    lambda: M.moe_route_topk(Tensor(f32, 8, 64), 4),
    lambda: M.moe_route_topk_backward(Tensor(f32, 8, 64), Tensor(i32, 8, 4), Tensor(f32, 8, 4)),
    lambda: M.mxfp4_quantize_rows(Tensor(bf16, 8, 64)),
    lambda: M.mxfp4_dequantize_rows(Tensor(u8, 128, 32), Tensor(u8, 512), 8, 64),
    lambda: M.mxfp4_quantize_weight(Tensor(bf16, 8, 64)),
    lambda: M.nvfp4_quantize_weight(Tensor(bf16, 8, 64)),
    lambda: M.mxfp4_linear(Tensor(bf16, 8, 64), M.FP4Weight(Tensor(u8, 128, 32), Tensor(u8, 512), None, 8, 64)),
    lambda: M.nvfp4_linear(Tensor(bf16, 8, 64), M.FP4Weight(Tensor(u8, 128, 32), Tensor(u8, 512), Tensor(f32, 8), 8, 64)),
    lambda: M.nvfp4_quantize_rows(Tensor(bf16, 8, 64)),
    lambda: M.nvfp4_silu_table(Tensor(f32, 65536)),
    lambda: M.moe_router_topk(Tensor(bf16, 8, 256), Tensor(bf16, 16, 256), 2),
    lambda: M.moe_route_sort_amax(Tensor(bf16, 8, 256), Tensor(i32, 8, 2), Tensor(f32, 8, 2), 4, Tensor(i32, 5), Tensor(u8, 8)),
    lambda: M.moe_expert_forward_nvfp4(weights(), 8, 2, Tensor(i32, 5), Tensor(bf16, 8, 256), Tensor(u8, 8)),
    lambda: weights().ref(),
    lambda: M.MoEWeightsBF16(Tensor(bf16, 4, 256, 256), Tensor(bf16, 4, 256, 128)).ref(),
], ids=["route_topk", "route_topk_backward", "mxfp4_quantize_rows", "mxfp4_dequantize_rows", "mxfp4_quantize_weight",
        "nvfp4_quantize_weight", "mxfp4_linear", "nvfp4_linear", "nvfp4_quantize_rows", "silu_table", "router_topk",
        "route_sort", "expert_forward", "expert_weights", "bf16_weights"])
def test_tensors_of_another_device(call):
    with pytest.raises(ValueError, match="current device"):
        call()


def test_stream_of_another_device():
    with pytest.raises(ValueError, match="current device"):
        M._stream(Stream(1))
    with pytest.raises(ValueError, match="current device"):
        M._raw_stream(Stream(1), Tensor(f32, 1))
    assert M._stream(Stream(0)).value is None and M._raw_stream(Stream(0), Tensor(f32, 1)) == 0
