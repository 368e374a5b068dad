"""One MoE block as a model has it: router, routed experts, a shared expert beside them, and the
gradient back through the routing.

    python examples/moe_block.py [--tokens T]

The router's scores are sigmoids, a bias that follows the experts' load takes part in the choice
only, and the experts of a token come from a few groups.  The routed experts run in the NVFP4
layer, the shared expert through two dense 4-bit products.
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
    """y = sum_j w_j expert_{id_j}(x) + shared(x)."""

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

    def shared(self, x):
        gate, up = M.nvfp4_linear(x, self.shared_up).float().chunk(2, dim=1)
        return M.mxfp4_linear((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), self.shared_down)

    def forward(self, x, train=False):
        _, _, logits = M.moe_router_topk(x, self.w_router, 1, with_logits=True)
        ids, w = M.moe_route_topk(logits, self.k, bias=self.bias, **self.route)
        self.saved = (x, logits, ids)
        return self.experts.forward(x, ids, w, save_for_backward=train) + self.shared(x)

    def backward(self, dout):
        """Gradients of the routed path: (dx, dw1, dw2 of the experts, dw_router)."""
        x, logits, ids = self.saved
        dx, dw1, dw2, dprob = self.experts.backward(dout)
        dlogits = M.moe_route_topk_backward(logits, ids, dprob, score="sigmoid", scale=self.route["scale"])
        dx = dx + (dlogits @ self.w_router.float()).to(torch.bfloat16)
        return dx, dw1, dw2, dlogits.t() @ x.float()

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
    for step in range(3):
        y = block.forward(x, train=True)
        dx, dw1, dw2, dw_router = block.backward(torch.ones_like(y))
        load = block.balance(step=0.01)
        print(f"step {step}: |y| {float(y.float().norm()):.3f}  |dx| {float(dx.float().norm()):.3f}  "
              f"|dw_router| {float(dw_router.norm()):.3f}  tokens per expert {int(load.min())}..{int(load.max())}")
    one = block.forward(x[:1])                                # serving: a single token
    print("one token equals its row of the batch:", bool(torch.equal(one, block.forward(x)[:1])))
    if M.nvfp4_get_device_error() != M.NVFP4_OK:
        raise RuntimeError("device error")


if __name__ == "__main__":
    main()
