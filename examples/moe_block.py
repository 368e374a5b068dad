"""One MoE block as a model has it: router, routed experts, a shared expert beside them with the
requests' own low-rank adapters, and the gradients of the router and the adapters.

    python examples/moe_block.py [--tokens T]

The router's scores are sigmoids, a bias that follows the experts' load takes part in the choice
only, a balance loss over each sequence keeps that choice even, and the experts of a token come
from a few groups.  The routed experts run in the NVFP4 layer, the shared expert through two dense
4-bit products, to the second of which each request adds the adapter it was trained with.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import nvfp4_moe_expert_gb300 as M  # noqa: E402


class MoEBlock:
    """y = sum_j w_j expert_{id_j}(x) + shared(x), shared(x) = down(act(x)) + scale_a B_a A_a act(x) with a
    token's adapter a."""

    def __init__(self, H, I, E, k, n_group, topk_group, scale=2.5, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape):
            return (0.02 * torch.randn(*shape, device=device, generator=g)).to(torch.bfloat16)

        self.k, self.E = k, E
        self.route = dict(score="sigmoid", n_group=n_group, topk_group=topk_group, group_score="top2", scale=scale)
        self.w_router = weight(E, H)
        self.bias = torch.zeros(E, device=device)
        self.experts = M.MoELayer(weight(E, 2 * I, H), weight(E, H, I))
        self.shared_up = M.nvfp4_quantize_weight(weight(2 * I, H))       # gate rows, then up rows
        self.shared_down = M.mxfp4_quantize_weight(weight(H, I))
        self.adapters, self.saved_shared = None, None

    def add_adapters(self, down, up, scale=None):
        """Adapters of the shared expert's second product: down [L, R, I], up [L, H, R], scale [L]."""
        self.adapters = M.LoRAAdapters(down, up, scale)

    def shared(self, x, adapter_ids=None, train=False):
        gate, up = M.nvfp4_linear(x, self.shared_up).float().chunk(2, dim=1)
        act = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
        y = M.mxfp4_linear(act, self.shared_down)
        if adapter_ids is None:
            return y
        if not train:
            return M.lora_add(y, act, self.adapters, adapter_ids, out=y)
        y, h = M.lora_add(y, act, self.adapters, adapter_ids, out=y, save_for_backward=True)
        self.saved_shared = (act, h, adapter_ids)
        return y

    def forward(self, x, train=False, adapter_ids=None):
        """adapter_ids: int32 [T], the adapter of each token's request (negative: none)."""
        _, _, logits = M.moe_router_topk(x, self.w_router, 1, with_logits=True)
        ids, w = M.moe_route_topk(logits, self.k, bias=self.bias, **self.route)
        self.saved = (x, logits, ids)
        return self.experts.forward(x, ids, w, save_for_backward=train) + self.shared(x, adapter_ids, train)

    def balance_loss(self, seq_offsets=None):
        """The balance loss of each sequence (int32 [S + 1] row offsets), and its counts, for backward."""
        _, logits, ids = self.saved
        return M.moe_balance_loss(logits, ids, score="sigmoid", seq_offsets=seq_offsets)

    def backward(self, dout, balance=None, weight=0.0, seq_offsets=None):
        """Gradients of the routed path, with `weight` times the sum of balance's losses: (dx, dw1, dw2 of the
        experts, dw_router)."""
        x, logits, ids = self.saved
        dx, dw1, dw2, dprob = self.experts.backward(dout)
        dlogits = M.moe_route_topk_backward(logits, ids, dprob, score="sigmoid", scale=self.route["scale"])
        if balance is not None:
            M.moe_balance_loss_backward(logits, self.k, balance.counts, balance.tokens, torch.full_like(balance.loss, weight),
                                        score="sigmoid", seq_offsets=seq_offsets, dlogits=dlogits)
        dx = dx + (dlogits @ self.w_router.float()).to(torch.bfloat16)
        return dx, dw1, dw2, dlogits.t() @ x.float()

    def adapter_gradients(self, dout):
        """Gradients of the adapters, the shared expert's own weights being fixed: (ddown, dup)."""
        act, h, adapter_ids = self.saved_shared
        return M.lora_add_backward(dout, act, h, self.adapters, adapter_ids)[1:]

    def balance(self, step=0.001):
        """Move the bias towards the experts that got fewer tokens than the mean."""
        load = torch.bincount(self.saved[2].flatten(), minlength=self.E).float()
        self.bias += step * torch.sign(load.mean() - load)
        return load


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    block = MoEBlock(H=512, I=256, E=64, k=6, n_group=8, topk_group=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(a.tokens, 512, device="cuda", generator=g).to(torch.bfloat16)
    block.add_adapters(0.02 * torch.randn(4, 16, 256, device="cuda", generator=g).to(torch.bfloat16),
                       0.02 * torch.randn(4, 512, 16, device="cuda", generator=g).to(torch.bfloat16))
    # four requests, one of them without an adapter; each is a sequence of its own for the balance loss
    seq_offsets = torch.linspace(0, a.tokens, 5, device="cuda").to(torch.int32)
    owner = torch.tensor([2, -1, 0, 3], dtype=torch.int32, device="cuda")
    adapter_ids = owner.repeat_interleave(seq_offsets.diff().long())
    for step in range(3):
        y = block.forward(x, train=True, adapter_ids=adapter_ids)
        balance = block.balance_loss(seq_offsets)
        dout = torch.ones_like(y)
        dx, dw1, dw2, dw_router = block.backward(dout, balance, weight=0.01, seq_offsets=seq_offsets)
        ddown, dup = block.adapter_gradients(dout)
        load = block.balance(step=0.01)
        print(f"step {step}: |y| {float(y.float().norm()):.3f}  |dx| {float(dx.float().norm()):.3f}  "
              f"|dw_router| {float(dw_router.norm()):.3f}  |ddown| {float(ddown.norm()):.3f}  |dup| {float(dup.norm()):.3f}  "
              f"balance loss {float(balance.loss.mean()):.3f}  tokens per expert {int(load.min())}..{int(load.max())}")
    one = block.forward(x[:1], adapter_ids=adapter_ids[:1])   # serving: a single token
    print("one token equals its row of the batch:", bool(torch.equal(one, block.forward(x, adapter_ids=adapter_ids)[:1])))
    if M.nvfp4_get_device_error() != M.NVFP4_OK:
        raise RuntimeError("device error")


if __name__ == "__main__":
    main()
