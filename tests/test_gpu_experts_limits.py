"""The expert operators at their limits: plans that no sort made, the widest
rows, calls that cannot be differentiated or traced as asked, and the accuracy
of what is rounded on the way."""
import math

import pytest
import torch

import expert_reference as R

pytestmark = pytest.mark.gpu

L = pytest.importorskip("differentiable_exact_budget_amd")


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradients_of_overlapping_experts_stay_in_bounds(dtype, act):
    """Offsets that run back: every other expert claims all rows, four times
    the row tiles that the scratch of the bias gradient has rows for.  A tile
    has 64 rows and there are 4096 / 64 + 8 + 1 = 73: expert 0 takes 64 of
    them, expert 2 the other 9, and none are left."""
    P, E, K, F, tiles = 4096, 8, 16, 24, 73
    off = torch.tensor([0, P] * (E // 2) + [0], dtype=torch.int32)
    plan = L.ExpertPlan(E, off.cuda(), torch.zeros(P, dtype=torch.int32).cuda(),
                        torch.zeros(P // 2, 2, dtype=torch.int32).cuda())
    g = gen(7)
    xs, dys = (torch.randn(P, n, generator=g).to(dtype) for n in (K, F))
    weight = (torch.randn(1, F, K, generator=g) * K ** -0.5).to(dtype).expand(E, F, K).contiguous()
    xsd, wd, dyd = xs.cuda(), weight.cuda(), dys.cuda()
    # z from a plan of one expert with all rows: the weights are all alike
    one = L.ExpertPlan(1, torch.tensor([0, P], dtype=torch.int32).cuda(), plan.order, plan.place)
    _, z = L.expert_linear_forward(xsd, wd[:1], one, activation=act)
    dx, dw, db = L.expert_linear_vjp(xsd, wd, plan, z, dyd, activation=act)
    assert dx.shape == xs.shape
    ref = R.linear(xs, weight[:1], None, torch.tensor([0, P]), act, dys)
    for e in range(E):
        R.check(dw[e:e + 1], *(t if e % 2 == 0 else torch.zeros_like(t) for t in ref["dw"]), f"dw of expert {e}")
    part = R.linear(xs[:64 * (tiles - 64)], weight[:1], None, torch.tensor([0, 64 * (tiles - 64)]), act,
                    dys[:64 * (tiles - 64)])
    for e in range(E):
        value, tol = ref["db"] if e == 0 else part["db"] if e == 2 else [torch.zeros_like(t) for t in ref["db"]]
        R.check(db[e:e + 1], value, tol, f"db of expert {e}")


WIDEST = 0x7FFF0000


@pytest.mark.slow
def test_more_tiles_than_32_bits_count():
    """One row among 32 experts of the widest outputs: tiles are counted with
    one more for each expert, 33 x 2^26 of 32 columns.  The sum is empty, so y
    is the zeros that the product writes."""
    E = 32
    plan = L.expert_sort(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), E)
    xs = torch.empty(1, 0, dtype=torch.bfloat16, device="cuda")
    weight = torch.empty(E, WIDEST, 0, dtype=torch.bfloat16, device="cuda")
    dirty = torch.full((1, WIDEST), math.nan, dtype=torch.bfloat16, device="cuda")
    del dirty  # y gets this memory
    y = L.expert_linear(xs, weight, plan)
    assert y.shape == (1, WIDEST)
    assert not y.any()
    del y
    torch.cuda.empty_cache()
