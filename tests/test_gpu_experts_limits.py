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


@pytest.mark.slow
def test_products_of_the_widest_outputs():
    """One row of one number to as many outputs as there may be, and back: each
    result is one product of two bf16, rounded once."""
    g = torch.Generator(device="cuda").manual_seed(3)
    plan = L.expert_sort(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    x = torch.full((1, 1), 1.5, dtype=torch.bfloat16, device="cuda")
    weight, dys = (torch.empty(WIDEST, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    y = L.expert_linear(x, weight.view(1, -1, 1), plan)
    assert torch.equal(y[0], weight * x[0])
    del y
    _, dw, db = L.expert_linear_vjp(x, weight.view(1, -1, 1), plan, None, dys.view(1, -1), want=(False, True, True))
    assert torch.equal(dw.view(-1), dys * x[0])
    assert torch.equal(db[0], dys)
    del weight, dys, dw, db
    torch.cuda.empty_cache()


@pytest.mark.slow
def test_the_widest_rows_to_their_places_and_back():
    D = 2 ** 31 - 1
    g = torch.Generator(device="cuda").manual_seed(4)
    plan = L.expert_sort(torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), 2)
    x = torch.empty(1, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    xs = L.expert_dispatch(x, plan)
    assert torch.equal(xs[0], x[0]) and torch.equal(xs[1], x[0])
    w = torch.tensor([[2.0, 0.5]], device="cuda")
    out = L.expert_combine(xs, w, plan, residual=x)
    assert torch.equal(out, x * 3.5)  # fp32 sums of multiples of x, exact
    del out
    # slot 0 is expert 1's row, behind expert 0's
    dys, _ = L.expert_combine_vjp(xs, w, plan, x, want=(True, False))
    assert torch.equal(dys[1], 2 * x[0]) and torch.equal(dys[0], 0.5 * x[0])
    del dys
    assert torch.equal(L.expert_dispatch_vjp(xs, plan), 2 * x)
    # dw: marks at a row's ends and middle, so that the sum is exact
    xs.zero_()
    at = torch.tensor([0, 1, D // 2, D - 2, D - 1], device="cuda")
    xs[0, at] = 1.0
    xs[1, at] = 2.0
    x.fill_(1.0)
    _, dw = L.expert_combine_vjp(xs, w, plan, x, want=(False, True))
    assert torch.equal(dw, torch.tensor([[10.0, 5.0]], device="cuda"))
    del x, xs
    torch.cuda.empty_cache()


def small_layer(dtype=torch.float32):
    """{operator: (call, its tensors that have a gradient)}"""
    g = gen(11)
    T, m, E, K, F = 6, 2, 4, 16, 24
    p = torch.rand(T, E, generator=g).cuda()
    plan = L.expert_sort(L.expert_topk(p, m)[0], E)
    x, xs, ys, res = (torch.randn(n, k, generator=g).to(dtype).cuda() for n, k in ((T, K), (T * m, K), (T * m, F), (T, F)))
    weight, bias = torch.randn(E, F, K, generator=g).to(dtype).cuda(), torch.randn(E, F, generator=g).to(dtype).cuda()
    w = torch.rand(T, m, generator=g).cuda()
    return {
        "expert_topk": (lambda p: L.expert_topk(p, m, normalize=True)[1], (p,)),
        "expert_dispatch": (lambda x: L.expert_dispatch(x, plan), (x,)),
        "expert_linear": (lambda xs, weight, bias: L.expert_linear(xs, weight, plan, bias=bias, activation="silu"),
                          (xs, weight, bias)),
        "expert_combine": (lambda ys, w, res: L.expert_combine(ys, w, plan, residual=res), (ys, w, res)),
    }


OPERATORS = ["expert_topk", "expert_dispatch", "expert_linear", "expert_combine"]


@pytest.mark.parametrize("name", OPERATORS)
@pytest.mark.parametrize("requires_grad", [False, True])
def test_forward_mode_derivatives_are_refused(name, requires_grad):
    """A tangent that an operator cannot carry on is not dropped: the call is refused, for each of its inputs."""
    fw = torch.autograd.forward_ad
    call, inputs = small_layer()[name]
    inputs = [t.detach().requires_grad_(requires_grad) for t in inputs]
    want = call(*inputs).detach()
    with fw.dual_level():
        for i in range(len(inputs)):
            dual = [fw.make_dual(t, torch.ones_like(t)) if i == j else t for j, t in enumerate(inputs)]
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(*dual)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
                call(*dual)
        assert torch.equal(call(*inputs), want)  # without tangents as ever


@pytest.mark.parametrize("name", OPERATORS + ["expert_sort"])
def test_traces_are_refused(name):
    """A trace would record the outputs' allocation and none of the work."""
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    call, inputs = small_layer()[name] if name != "expert_sort" else (lambda ids: L.expert_sort(ids, 3).order, (ids,))
    for grad in (False, True) if name != "expert_sort" else (False,):
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(call, tuple(t.detach().requires_grad_(grad) for t in inputs), check_trace=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gelu_keeps_its_relative_accuracy_far_below_zero(dtype):
    """For 16-bit rows gelu(z) = z Q(-z) with a polynomial Q that is 2.1e-4 Q
    off at most; its exponential's argument, below 122 here, is rounded twice
    (3e-5).  Then one rounding to the rows' type."""
    z = torch.cat([torch.linspace(-13, -4, 4096), torch.linspace(-4, 4, 4096), torch.linspace(4, 13, 64)]).to(dtype)
    F = z.numel()
    plan = L.expert_sort(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    y = L.expert_linear(torch.zeros(1, 16, dtype=dtype).cuda(), torch.zeros(1, F, 16, dtype=dtype).cuda(), plan,
                        bias=z[None].cuda(), activation="gelu")
    z = z.double()
    ref = 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    R.check(y[0], ref, R.rounded(ref, dtype, 2.4e-4 * ref.abs()), "gelu")


@pytest.mark.parametrize("name", ["expert_linear", "expert_combine"])
def test_only_what_the_wanted_gradients_read_is_kept(name):
    """dxs reads the weights, dweight the rows, the combined rows' gradient the
    gates and the gates' gradient the rows: what no wanted gradient reads is
    not kept between the passes, and the gradients are as with all wanted."""
    call, inputs = small_layer()[name]
    dout = torch.randn(call(*inputs).shape, generator=gen(5)).cuda()
    leaves = [t.detach().requires_grad_(True) for t in inputs]
    all_grads = torch.autograd.grad(call(*leaves), leaves, dout)
    readers = {"expert_linear": ((1,), (0,), ()), "expert_combine": ((), (0,), ())}[name]  # rows and weights
    for i in range(3):
        leaves = [t.detach().requires_grad_(i == j) for j, t in enumerate(inputs)]
        kept = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t.data_ptr()), t)[1], lambda t: t):
            out = call(*leaves)
        for j in range(3):
            if j == 1 and name == "expert_combine":
                continue  # the gates, a number for every row
            assert (inputs[j].data_ptr() in kept) == (j in readers[i]), (i, j)
        assert torch.equal(torch.autograd.grad(out, leaves[i], dout)[0], all_grads[i])
