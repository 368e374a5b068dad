"""Numbers that the C structs and arguments of the routing calls cannot hold are refused, not cut to 32 bits."""

import pytest
import torch

import nvfp4_moe_expert_gb300 as M

WRAPS = [(1 << 32) + 4, (1 << 31), -(1 << 32) + 4]


@pytest.mark.parametrize("value", WRAPS)
@pytest.mark.parametrize("which", ["k", "n_group", "topk_group"])
def test_parameters(which, value):
    kw = dict(score="softmax", k=4, n_group=4, topk_group=2, group_score="max", renormalize=True, scale=1.0)
    assert getattr(M._route_params(**kw), which) == kw[which]
    kw[which] = value
    with pytest.raises(ValueError, match=which):
        M._route_params(**kw)


@pytest.mark.parametrize("experts", [(1 << 32) + 8, 1 << 31])
def test_experts(monkeypatch, experts):
    class Logits:
        dtype, device, is_cuda = torch.float16, torch.device("cuda", 0), True
        shape = torch.Size((1, experts))

        def dim(self):
            return 2

        def stride(self):
            return experts, 1

        def get_device(self):
            return 0

    monkeypatch.setattr(M, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="experts"):
        M.moe_route_topk(Logits(), 4)
    with pytest.raises(ValueError, match="experts"):
        M.moe_route_topk_backward(Logits(), torch.zeros((1, 4), dtype=torch.int32), torch.zeros((1, 4)))
