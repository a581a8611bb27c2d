"""A routed layer trained on the GPU: every token's scores become gates with an
exact budget, its m largest gates choose its experts, and the experts' outputs
come back weighted by them.

    p = soft_topk_rows(scores, m, t)          sum over a row: m exactly
    ids, w = expert_topk(p, m)                the m largest gates
    plan = expert_sort(ids, experts)          pairs in expert order
    h = expert_linear(expert_dispatch(x, plan), w1, plan, bias=b1, activation="gelu")
    out = expert_combine(expert_linear(h, w2, plan), w, plan, residual=x)

Fits a fixed random layer of the same shape and prints the loss and each
expert's share of the tokens.

    python examples/expert_block.py [--steps 200] [--tokens 2048] [--experts 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import differentiable_exact_budget_amd as L  # noqa: E402


class ExpertBlock(torch.nn.Module):
    """x + the weighted outputs of m of the experts, two layers each."""

    def __init__(self, width: int, hidden: int, experts: int, m: int, t: float = 0.3, dtype=torch.bfloat16,
                 device="cuda", generator=None):
        super().__init__()
        self.experts, self.m, self.t = experts, m, t

        def normal(*shape, fan, kind=dtype):
            x = torch.randn(*shape, generator=generator, device=device) * fan ** -0.5
            return torch.nn.Parameter(x.to(kind))

        self.router = normal(experts, width, fan=width, kind=torch.float32)
        self.w1 = normal(experts, hidden, width, fan=width)
        self.b1 = torch.nn.Parameter(torch.zeros(experts, hidden, dtype=dtype, device=device))
        self.w2 = normal(experts, width, hidden, fan=hidden)

    def route(self, x: torch.Tensor):
        """(plan, weights): the gates of a row sum to m, so a weight is the
        share of its slot that the router spends on the expert."""
        p = L.soft_topk_rows(x.float() @ self.router.t(), float(self.m), self.t)
        ids, w = L.expert_topk(p, self.m)
        return L.expert_sort(ids, self.experts), w

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        plan, w = self.route(x)
        h = L.expert_linear(L.expert_dispatch(x, plan), self.w1, plan, bias=self.b1, activation="gelu")
        return L.expert_combine(L.expert_linear(h, self.w2, plan), w, plan, residual=x)


def train(steps: int = 200, tokens: int = 2048, experts: int = 8, m: int = 2, width: int = 256, hidden: int = 512,
          lr: float = 2e-3, seed: int = 0, report=print):
    """The losses of `steps` steps of Adam on the layer's weights in fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher = ExpertBlock(width, hidden, experts, m, generator=g)
    layer = ExpertBlock(width, hidden, experts, m, dtype=torch.float32, generator=g)
    layer.router.data.copy_(teacher.router.data + 0.02 * torch.randn(teacher.router.shape, generator=g, device="cuda"))
    opt = torch.optim.Adam(layer.parameters(), lr=lr)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda")
        with torch.no_grad():
            target = teacher(x.bfloat16()).float()
        loss = (layer(x) - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % max(1, steps // 10) == 0 or step == steps - 1:
            losses.append(loss.item())
            report(f"step {step:4d}  loss {losses[-1]:.4f}")
    plan, _ = layer.route(x)
    share = (plan.offsets[1:] - plan.offsets[:-1]).float() / plan.offsets[-1]
    report("share of the pairs: " + " ".join(f"{s:.3f}" for s in share.tolist()))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.experts)
