"""The routed layer of examples/expert_block.py: its forward pass and every
gradient against the same layer in float64 operations, and a short training."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

L = pytest.importorskip("differentiable_exact_budget_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from expert_block import ExpertBlock, train  # noqa: E402


def test_layer_and_gradients_against_float64():
    T, width, hidden, E, m, t = 40, 32, 48, 6, 2, 0.3
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = ExpertBlock(width, hidden, E, m, t, dtype=torch.float32, generator=g)
    layer.b1.data.normal_(generator=g)
    x = torch.randn(T, width, generator=g, device="cuda", requires_grad=True)
    c = torch.randn(T, width, generator=g, device="cuda")
    out = layer(x)
    (out * c).sum().backward()

    # the same in float64: the budget's threshold by bisection, then as a
    # function of the scores through its own implicit gradient
    xd = x.detach().double().requires_grad_(True)
    router, w1, b1, w2 = (p.detach().double().requires_grad_(True) for p in (layer.router, layer.w1, layer.b1, layer.w2))
    r = xd @ router.t()
    cdf = lambda z: torch.where(z < 0, 0.5 * torch.exp(z), 1 - 0.5 * torch.exp(-z.abs()))  # noqa: E731
    with torch.no_grad():
        lo, hi = r.min(1, keepdim=True).values - 20 * t, r.max(1, keepdim=True).values + 20 * t
        for _ in range(200):
            b = 0.5 * (lo + hi)
            more = cdf((r - b) / t).sum(1, keepdim=True) > m
            lo, hi = torch.where(more, b, lo), torch.where(more, hi, b)
        f = 0.5 * torch.exp(-(r - b).abs() / t)
    b = b + ((f / f.sum(1, keepdim=True)) * (r - r.detach())).sum(1, keepdim=True)  # db/dr_i = f_i / sum f
    p = cdf((r - b) / t)
    ids = L.expert_topk(L.soft_topk_rows((x.detach() @ layer.router.detach().t()), float(m), t), m)[0].long()
    w = p.gather(1, ids)
    h = torch.nn.functional.gelu(torch.einsum("td,tjhd->tjh", xd, w1[ids]) + b1[ids])
    ref = xd + (torch.einsum("tjh,tjdh->tjd", h, w2[ids]) * w[:, :, None]).sum(1)
    (ref * c.double()).sum().backward()
    # fp32 sums of at most 48 terms of order 1 in a chain of six operations, and
    # gates within 2e-6: 1e-4 of the largest value holds with room
    for name, a, e in (("out", out, ref), ("x", x.grad, xd.grad), ("router", layer.router.grad, router.grad),
                       ("w1", layer.w1.grad, w1.grad), ("b1", layer.b1.grad, b1.grad), ("w2", layer.w2.grad, w2.grad)):
        err = (a.detach().double() - e).abs().max().item()
        assert err <= 1e-4 * max(1.0, e.abs().max().item()), f"{name}: {err}"


def test_training_lowers_the_loss():
    losses = train(steps=40, tokens=512, experts=4, width=64, hidden=128, report=lambda s: None)
    assert losses[-1] < 0.7 * losses[0], losses
