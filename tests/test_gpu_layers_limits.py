"""The norm, the loss and the experts' products in 8 bits at their limits: rows
that take no part and hold anything, results of nothing, and sizes that take the
kernels' rarer paths."""
import math

import pytest
import torch

from test_gpu_layers import L, TYPES, gen, loss_case

pytestmark = pytest.mark.gpu


# ---- rows that take no part in a loss ------------------------------------------------

def spoiled(x, rows):
    """x with NaN, infinities and the type's largest values in some rows."""
    x = x.clone()
    kinds = (math.nan, math.inf, -math.inf, torch.finfo(x.dtype).max)
    for i, r in enumerate(rows):
        x[r, i % x.shape[1]:] = kinds[i % 4]
    return x


# few rows; tiles that share dx's sum and that do not; the widest for d, dx and dW;
# odd widths on narrow and on wide tiles
@pytest.mark.parametrize("T,V,D", [(20, 200, 64), (50, 200, 64), (300, 3000, 136), (1040, 600, 2048), (3100, 4001, 64),
                                   (100, 16384, 768), (20, 200, 33), (50, 200, 33), (1100, 2100, 129)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_a_gradient_may_hold_anything(T, V, D, dtype):
    """Ignored rows, and rows whose loss has the gradient 0: every gradient is
    the one with zeros in their place."""
    x, w, b, target = loss_case(T, V, D, dtype, drop=0.0)
    out, still = torch.arange(1, T, 7), torch.arange(3, T, 7)
    target[out[0::2]], target[out[1::2]] = -100, V
    clean = x.clone()
    clean[out], clean[still] = 0, 0
    bad = spoiled(x, torch.cat([out, still]).tolist())
    dloss = torch.rand(T, generator=gen(4)) + 0.5
    dloss[still] = 0
    got = []
    for rows in (bad, clean):
        leaves = [t.cuda().requires_grad_(True) for t in (rows, w, b)]
        loss = L.linear_cross_entropy(leaves[0], leaves[1], target.cuda(), bias=leaves[2], reduction="none")
        got.append(torch.autograd.grad(loss, leaves, dloss.cuda()))
    for name, a, c in zip(("dx", "dw", "db"), *got):
        assert a.isfinite().all() and torch.equal(a, c), name
    assert got[0][0][out].abs().max() == 0 and got[0][0][still].abs().max() == 0
    assert got[0][0].abs().max() > 0 and got[0][1].abs().max() > 0


@pytest.mark.parametrize("T,V,D", [(20, 200, 64), (300, 600, 136), (1040, 600, 2048), (50, 200, 33), (1100, 2100, 129)])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_without_a_gradient_have_none_whatever_the_weights_hold(T, V, D, dtype):
    x, w, b, target = loss_case(T, V, D, dtype, drop=0.3)
    w[5, 3], w[V - 1, 0] = math.nan, math.inf
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    L.linear_cross_entropy(leaves[0], leaves[1], target.cuda(), bias=leaves[2]).backward()
    none = target < 0
    assert leaves[0].grad[none].abs().max() == 0 and leaves[0].grad[~none].isnan().any(1).all()
