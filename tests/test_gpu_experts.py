"""The expert operators against their definitions in float64: the choice of
gates, the pair sort, dispatch, the experts' products and combine, forward and
backward, at the sizes, masks and alignments where they can go wrong.
Tolerances are the kernels' worst-case rounding (expert_reference)."""
import math

import pytest
import torch

import expert_reference as R

pytestmark = pytest.mark.gpu

L = pytest.importorskip("differentiable_exact_budget_amd")

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def some_ids(T, m, E, seed, drop=0.2, idle=()):
    g = gen(seed)
    score = torch.rand(T, E, generator=g)
    for e in idle:
        score[:, e] = -1
    ids = score.topk(min(m, E), dim=1).indices.int()
    if m > E:
        ids = torch.cat([ids, torch.full((T, m - E), -1, dtype=torch.int32)], 1)
    ids[torch.rand(T, m, generator=g) < drop] = -1
    for e in idle:
        ids[ids == e] = -1
    return ids


def make_plan(ids, E):
    o, order, place = R.sort(ids, E)
    return L.ExpertPlan(E, o.cuda(), order.cuda(), place.cuda()), o, order, place


# ---- topk --------------------------------------------------------------------

@pytest.mark.parametrize("T,E,m", [(1, 1, 1), (3, 5, 2), (17, 16, 16), (33, 17, 4), (8, 64, 4), (50, 65, 7),
                                   (100, 257, 8), (5, 300, 64), (9, 1024, 33), (1, 1024, 64), (0, 8, 2)])
@pytest.mark.parametrize("normalize", [False, True])
def test_topk(T, E, m, normalize):
    p = torch.rand(T, E, generator=gen(T + E + m))
    ref, w, sums = R.topk(p, m, normalize=normalize)
    pd = p.cuda().requires_grad_(True)
    ids, got = L.expert_topk(pd, m, normalize=normalize)
    assert torch.equal(ids.cpu(), ref)
    # normalized: m - 1 additions, one division
    R.check(got, w, w.abs() * R.EPS * (m + 1), "weights")
    dw = torch.randn(T, m, generator=gen(1))
    got.backward(dw.cuda())
    dp = R.topk_vjp(ref, w, sums, dw, E, normalize)
    big = dw.abs().double().amax(1, keepdim=True) if T else dw.double().sum(1, keepdim=True)
    tol = (4 * m + 8) * R.EPS * (big / sums[:, None] if normalize else big)
    R.check(pd.grad, dp, tol.expand(T, E), "dp")


def test_topk_ties_floors_and_unusual_values():
    inf, nan = math.inf, math.nan
    low = torch.finfo(torch.float32).min
    p = torch.tensor([
        [0.5, 0.5, 0.5, 0.5, 0.5],           # ties: the lowest experts
        [-0.0, 0.0, -0.0, 0.0, -1.0],        # zeros of either sign tie
        [nan, 1.0, nan, 2.0, nan],           # NaN is never chosen
        [-inf, -inf, -inf, -inf, -inf],      # nothing to choose
        [nan, nan, nan, nan, nan],
        [low, low, -inf, low, nan],          # the lowest finite value can be
        [inf, 1.0, 2.0, -inf, 3.0],
        [-3.0, -2.0, -1.0, -4.0, -5.0],      # a sum below 0
    ])
    for floor in (-inf, 0.25, 1.0, inf):
        ref, w, _ = R.topk(p, 3, floor=floor)
        ids, got = L.expert_topk(p.cuda(), 3, floor=floor)
        assert torch.equal(ids.cpu(), ref), floor
        assert torch.equal(got.cpu().double(), w), floor
    ids, w = L.expert_topk(p.cuda(), 3, normalize=True)
    w = w.cpu()
    assert torch.equal(w[3], torch.zeros(3)) and torch.equal(w[4], torch.zeros(3))
    assert torch.equal(w[7], torch.zeros(3)), "a sum that is not above 0 gives weights 0"
    assert torch.equal(ids.cpu()[7], torch.tensor([2, 1, 0], dtype=torch.int32))


def test_topk_gradient_of_empty_rows_and_zero_sums_is_zero():
    p = torch.tensor([[-math.inf] * 4, [-1.0, -2.0, -3.0, -4.0], [1.0, math.nan, -math.inf, 3.0]])
    pd = p.cuda().requires_grad_(True)
    ids, w = L.expert_topk(pd, 3, normalize=True)
    w.backward(torch.tensor([[1.0, 2.0, 3.0]] * 3).cuda())
    g = pd.grad.cpu()
    assert torch.equal(g[:2], torch.zeros(2, 4))
    # weights 3/4 and 1/4 of experts 3 and 0: d = (dw - 1.25) / 4
    assert torch.allclose(g[2], torch.tensor([0.1875, 0.0, 0.0, -0.0625]), rtol=0, atol=4 * R.EPS)


# ---- sort --------------------------------------------------------------------

@pytest.mark.parametrize("T,m,E,drop", [
    (0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 1, 1, 1.0), (5, 3, 8, 0.3), (8, 4, 64, 0.0), (64, 8, 257, 0.1),
    (1023, 4, 5, 0.0), (2048, 8, 1024, 0.5), (16385, 1, 3, 0.2),         # one workgroup, then many
    (5000, 8, 257, 0.1), (70001, 3, 1024, 0.1), (30000, 2, 64, 1.0), (700001, 8, 31, 0.05),
])
def test_sort(T, m, E, drop):
    if m <= E and T <= 20000:
        ids = some_ids(T, m, E, T + m, drop)
    else:
        g = gen(T)
        ids = torch.randint(0, E, (T, m), generator=g, dtype=torch.int32)
        ids[torch.rand(T, m, generator=g) < drop] = -1
    ref = R.sort(ids, E)
    plan = L.expert_sort(ids.cuda(), E)
    for name, a, b in zip(("offsets", "order", "place"), (plan.offsets, plan.order, plan.place), ref):
        assert torch.equal(a.cpu(), b), name


@pytest.mark.parametrize("T", [100, 20000])
def test_sort_one_expert_takes_all_and_ids_out_of_range_are_empty(T):
    ids = torch.full((T, 2), 6, dtype=torch.int32)
    ids[::3, 1] = 9            # outside the experts
    ids[1::3, 1] = -7
    ids[2::5, 0] = 2 ** 31 - 1
    ids[3::5, 0] = -2 ** 31
    ref = R.sort(ids, 9)
    plan = L.expert_sort(ids.cuda(), 9)
    for a, b in zip((plan.offsets, plan.order, plan.place), ref):
        assert torch.equal(a.cpu(), b)


# ---- dispatch and combine ----------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,m,E,D,drop", [(1, 1, 1, 1, 0.0), (1, 8, 64, 4096, 0.0), (7, 3, 5, 33, 0.4),
                                          (130, 2, 9, 1001, 0.2), (65, 4, 4, 520, 1.0), (257, 2, 8, 2048, 0.1),
                                          (3, 64, 70, 24, 0.5), (0, 2, 4, 16, 0.0), (5, 2, 4, 0, 0.0)])
def test_dispatch_and_combine(dtype, T, m, E, D, drop):
    ids = some_ids(T, m, E, T * 3 + D, drop)
    plan, o, order, place = make_plan(ids, E)
    g = gen(D + 5)
    x = torch.randn(T, D, generator=g).to(dtype)
    xd = x.cuda().requires_grad_(True)
    xs = L.expert_dispatch(xd, plan)
    assert torch.equal(xs.detach().cpu(), R.dispatch(x, order, m))
    dxs = torch.randn(T * m, D, generator=g).to(dtype)
    dxs[int(o[-1]):] = math.nan  # rows of no pair: not read
    xs.backward(dxs.cuda())
    rows = R.gather(dxs, place)
    ref = rows.sum(1)
    R.check(xd.grad, ref, R.rounded(ref, dtype, m * R.EPS * rows.abs().sum(1)), "dx")

    ys = torch.randn(T * m, D, generator=g).to(dtype)
    ys[int(o[-1]):] = math.nan
    w = torch.rand(T, m, generator=g)
    w[place < 0] = math.nan      # weights of empty slots: not used
    res = torch.randn(T, D, generator=g).to(dtype)
    rows = R.gather(ys, place)
    w0 = torch.where(place >= 0, w, torch.zeros(())).double()
    for residual in (None, res):
        yd, wd = ys.cuda().requires_grad_(True), w.cuda().requires_grad_(True)
        rd = residual.cuda().requires_grad_(True) if residual is not None else None
        out = L.expert_combine(yd, wd, plan, residual=rd)
        ref, mag = (rows * w0[:, :, None]).sum(1), (rows * w0[:, :, None]).abs().sum(1)
        if residual is not None:
            ref, mag = ref + residual.double(), mag + residual.double().abs()
        R.check(out, ref, R.rounded(ref, dtype, (m + 1) * R.EPS * mag), "out")
        dout = torch.randn(T, D, generator=gen(9)).to(dtype)
        out.backward(dout.cuda())
        d = dout.double()
        dys = torch.zeros(T * m, D).double()
        on = order >= 0
        pair = order[on].long()
        dys[on] = w0.reshape(-1)[pair][:, None] * d[pair // m]
        R.check(yd.grad, dys, R.rounded(dys, dtype, 2 * R.EPS * dys.abs()), "dys")
        dw = (rows * d[:, None, :]).sum(2)
        R.check(wd.grad, dw, (D + 2) * R.EPS * (rows * d[:, None, :]).abs().sum(2) + R.TINY[torch.float32], "dw")
        if residual is not None:
            assert torch.equal(rd.grad.cpu(), dout)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_off_16_bytes(dtype):
    """Rows whose width is a multiple of 16 bytes in tensors that do not start on one."""
    T, m, E, D = 40, 2, 6, 64
    plan, o, order, place = make_plan(some_ids(T, m, E, 1), E)
    flat = torch.randn(T * D + 1, generator=gen(2)).to(dtype).cuda()
    x = flat[1:].reshape(T, D)
    assert x.data_ptr() % 16 != 0 and x.is_contiguous()
    xs = L.expert_dispatch(x, plan)
    assert torch.equal(xs.cpu(), R.dispatch(x.cpu(), order, m))
    wt = torch.randn(E * 32 * D + 1, generator=gen(3)).to(dtype).cuda()[1:].reshape(E, 32, D)
    ref = R.linear(xs.cpu(), wt.cpu(), None, o, "none")
    R.check(L.expert_linear(xs, wt, plan), *ref["ys"], "ys")


def test_non_contiguous_inputs_are_laid_out_by_the_differentiable_calls():
    T, m, E, D = 30, 2, 6, 48
    plan, o, order, place = make_plan(some_ids(T, m, E, 1), E)
    x = torch.randn(D, T, generator=gen(2)).cuda().t()
    assert not x.is_contiguous()
    xs = L.expert_dispatch(x, plan)
    assert torch.equal(xs.cpu(), R.dispatch(x.cpu().contiguous(), order, m))
    p = torch.rand(E, T, generator=gen(4)).cuda().t()
    ids, w = L.expert_topk(p, m)
    assert torch.equal(ids.cpu(), R.topk(p.cpu(), m)[0])
    wt = torch.randn(E, D, 40, generator=gen(5)).cuda().transpose(1, 2)
    R.check(L.expert_linear(xs, wt, plan), *R.linear(xs.cpu(), wt.cpu(), None, o, "none")["ys"], "ys")
    # an expanded upstream gradient
    out = L.expert_combine(xs.requires_grad_(True), torch.ones(T, m, device="cuda"), plan)
    out.sum().backward()
    assert torch.equal(xs.grad.cpu(), (order >= 0).float()[:, None].expand(T * m, D))


# ---- the experts' products ---------------------------------------------------

def product_case(dtype, T, m, E, K, F, act, bias=True, drop=0.1, idle=(), seed=0):
    ids = some_ids(T, m, E, seed + T, drop, idle)
    plan, o, order, place = make_plan(ids, E)
    g = gen(seed + K * F)
    P = T * m
    if act == "relu":  # whole numbers, and a half from the bias: z is exact and never 0
        xs = torch.randint(-2, 3, (P, K), generator=g).to(dtype)
        weight = torch.randint(-1, 2, (E, F, K), generator=g).to(dtype)
        b = (torch.randint(0, 2, (E, F), generator=g) - 0.5).to(dtype)
    else:
        xs = torch.randn(P, K, generator=g).to(dtype)
        weight = (torch.randn(E, F, K, generator=g) * max(K, 1) ** -0.5).to(dtype)
        b = torch.randn(E, F, generator=g).to(dtype)
    dys = torch.randn(P, F, generator=g).to(dtype)
    used = int(o[-1])
    xs[used:] = math.nan          # not read
    dys[used:] = math.nan
    for e in range(E):
        if o[e] == o[e + 1]:
            weight[e] = math.nan  # an expert without rows: not read into any result
    return plan, o, xs, weight, b if bias else None, dys, used


def check_product(dtype, T, m, E, K, F, act, bias=True, on="cpu", **kw):
    plan, o, xs, weight, b, dys, used = product_case(dtype, T, m, E, K, F, act, bias, **kw)
    leaves = [t.cuda().requires_grad_(True) for t in (xs, weight, b) if t is not None]
    y = L.expert_linear(leaves[0], leaves[1], plan, bias=leaves[2] if bias else None, activation=act)
    xs0, dys0, w0 = xs.clone(), dys.clone(), weight.clone()
    xs0[used:] = 0
    dys0[used:] = 0
    ref = R.linear(*(None if t is None else t.to(on) for t in (xs0, w0, b)), o, act, dys0.to(on))
    R.check(y, *ref["ys"], "ys")
    with torch.no_grad():  # the serving call keeps no z
        y1 = L.expert_linear(leaves[0], leaves[1], plan, bias=leaves[2] if bias else None, activation=act)
    assert torch.equal(y1, y)
    y.backward(dys.cuda())
    for name, t in zip(("dxs", "dw", "db"), leaves):
        R.check(t.grad, *ref[name], name)


SIZES = [
    (1, 1, 1, 1, 1), (1, 2, 4, 64, 64), (3, 1, 2, 7, 5), (4, 4, 64, 128, 96), (33, 2, 3, 65, 63), (100, 2, 7, 257, 130),
    (64, 2, 4, 72, 200), (300, 2, 5, 128, 256), (520, 1, 2, 320, 264), (700, 2, 3, 512, 520), (16, 4, 16, 1024, 512),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,m,E,K,F", SIZES)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_products(dtype, T, m, E, K, F, act):
    check_product(dtype, T, m, E, K, F, act, idle=(1,) if E > 3 else ())


# enough rows for every tile size, ends inside the tiles, and widths off 16
# bytes; the float64 reference runs on the GPU
LARGE = [(2000, 2, 12, 520, 520), (8000, 2, 5, 1032, 4104), (4000, 2, 8, 1001, 2001), (1500, 2, 4, 1024, 513),
         (700, 2, 5, 2056, 264)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,m,E,K,F", LARGE)
def test_products_of_many_rows(dtype, T, m, E, K, F):
    check_product(dtype, T, m, E, K, F, "silu", idle=(2,), on="cuda")


# many rows narrower than 16 bytes on one side or both, and up to four rows of
# each expert over long sums with a masked end
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,m,E,K,F", [(20000, 2, 3, 5, 7), (20000, 2, 3, 3, 600), (20000, 2, 3, 600, 3),
                                       (16, 4, 16, 1032, 200), (40, 2, 24, 1048, 40), (9, 4, 9, 2047, 33)])
def test_products_of_narrow_rows_and_of_few_rows(dtype, T, m, E, K, F):
    check_product(dtype, T, m, E, K, F, "silu", idle=(1,), on="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("T,m,E,K,F", [(50, 2, 4, 64, 128), (21, 3, 5, 33, 40), (300, 2, 3, 256, 264)])
def test_products_other_activations(dtype, T, m, E, K, F, act):
    check_product(dtype, T, m, E, K, F, act)


@pytest.mark.parametrize("dtype", TYPES)
def test_products_without_bias_and_with_all_rows_of_one_expert(dtype):
    check_product(dtype, 300, 1, 3, 136, 72, "gelu", bias=False, idle=(0, 2), drop=0.0)
    check_product(dtype, 600, 1, 1, 64, 320, "none", bias=False, drop=0.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_products_of_empty_plans_and_widths(dtype):
    E, F, K = 3, 40, 24
    weight = torch.full((E, F, K), math.nan, dtype=dtype).cuda().requires_grad_(True)
    bias = torch.full((E, F), math.nan, dtype=dtype).cuda().requires_grad_(True)
    for T, ids in ((4, torch.full((4, 2), -1, dtype=torch.int32)), (0, torch.empty(0, 2, dtype=torch.int32))):
        plan = L.expert_sort(ids.cuda(), E)
        xs = torch.full((T * 2, K), math.nan, dtype=dtype).cuda().requires_grad_(True)
        y = L.expert_linear(xs, weight, plan, bias=bias, activation="silu")
        assert torch.equal(y.detach(), torch.zeros(T * 2, F, dtype=dtype, device="cuda"))
        y.backward(torch.full_like(y, math.nan))
        for t in (xs, weight, bias):
            assert torch.equal(t.grad, torch.zeros_like(t)), T
            t.grad = None
    ids = torch.tensor([[0, 2], [1, -1]], dtype=torch.int32)
    plan = L.expert_sort(ids.cuda(), E)
    b = torch.randn(E, F, generator=gen(1)).to(dtype).cuda()
    y = L.expert_linear(torch.empty(4, 0, dtype=dtype).cuda(), torch.empty(E, F, 0, dtype=dtype).cuda(), plan, bias=b)
    assert torch.equal(y, torch.cat([b, torch.zeros(1, F, dtype=dtype, device="cuda")]))
    xs = torch.randn(4, K, generator=gen(2)).to(dtype).cuda().requires_grad_(True)
    y = L.expert_linear(xs, torch.empty(E, 0, K, dtype=dtype).cuda(), plan)
    assert y.shape == (4, 0)
    y.sum().backward()
    assert torch.equal(xs.grad, torch.zeros_like(xs))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes_at_extreme_z(dtype, act):
    """z far outside fp16 and relu's z too small for it."""
    z = torch.tensor([[-6e4, 6e4, 1e-9, -1e-9, 0.0, 3.0, -3.0, 1e-30]]).to(dtype)
    if dtype == torch.bfloat16:
        z = torch.cat([z, torch.tensor([[1e30, -1e30, 7e4, -7e4, 1e5, -1e5, 3e38, -3e38]]).to(dtype)], 1)
    F = z.shape[1]
    plan = L.expert_sort(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    xs = torch.zeros(1, 16, dtype=dtype).cuda()
    weight = torch.zeros(1, F, 16, dtype=dtype).cuda()
    bias = z.cuda().requires_grad_(True)
    y = L.expert_linear(xs, weight, plan, bias=bias, activation=act)
    z64 = z.double()
    ref = R.act(z64, act)
    R.check(y, ref, R.rounded(ref, dtype, 16 * R.EPS * z64.abs()), "ys")
    y.backward(torch.ones_like(y))
    s = R.slope(z64, act)
    R.check(bias.grad, s, R.rounded(s, dtype, 2.0 ** -11 * z64.abs().clamp(max=30) + 2.0 ** -20), "slopes")


def test_gradients_against_differences():
    """The whole chain in fp32 against central differences of its definition in float64."""
    T, E, m, K, F = 5, 4, 2, 6, 7
    g = gen(3)
    p, x = torch.rand(T, E, generator=g), torch.randn(T, K, generator=g)
    w1, b1 = torch.randn(E, F, K, generator=g) * 0.4, torch.randn(E, F, generator=g)
    w2, b2 = torch.randn(E, K, F, generator=g) * 0.4, torch.randn(E, K, generator=g)
    c = torch.randn(T, K, generator=g)
    leaves = [t.cuda().requires_grad_(True) for t in (p, x, w1, b1, w2, b2)]
    pd, xd, w1d, b1d, w2d, b2d = leaves
    ids, w = L.expert_topk(pd, m, normalize=True)
    plan = L.expert_sort(ids, E)
    h = L.expert_linear(L.expert_dispatch(xd, plan), w1d, plan, bias=b1d, activation="gelu")
    out = L.expert_combine(L.expert_linear(h, w2d, plan, bias=b2d, activation="silu"), w, plan, residual=xd)
    (out * c.cuda()).sum().backward()
    ids = ids.cpu().long()

    def loss(p, x, w1, b1, w2, b2):
        gate = p.gather(1, ids)
        gate = gate / gate.sum(1, keepdim=True)
        total = (x * c.double()).sum()
        for t in range(T):
            for j in range(m):
                e = int(ids[t, j])
                y = R.act(w2[e] @ R.act(w1[e] @ x[t] + b1[e], "gelu") + b2[e], "silu")
                total = total + gate[t, j] * (y * c[t].double()).sum()
        return total

    args = [t.double() for t in (p, x, w1, b1, w2, b2)]
    for k, leaf in enumerate(leaves):
        diff = torch.zeros_like(args[k])
        flat = diff.reshape(-1)
        for i in range(flat.numel()):
            step = []
            for h in (1e-5, -1e-5):
                moved = [a.clone() for a in args]
                moved[k].reshape(-1)[i] += h
                step.append(loss(*moved))
            flat[i] = (step[0] - step[1]) / 2e-5
        # fp32 chain of sums of at most 40 terms of order 1, differences exact to 1e-9
        R.check(leaf.grad, diff, torch.full_like(diff, 400 * R.EPS * float(diff.abs().max() + 1)), f"gradient {k}")


# ---- refusals, streams, graphs, long rows ------------------------------------

def test_refusals():
    dev = "cuda"
    p = torch.rand(4, 8, device=dev)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    plan = L.expert_sort(ids, 3)
    x = torch.randn(4, 16, device=dev)
    xs = L.expert_dispatch(x, plan)
    wt = torch.randn(3, 5, 16, device=dev)
    w = torch.rand(4, 2, device=dev)
    bad = [
        lambda: L.expert_topk(p.double(), 2), lambda: L.expert_topk(p, 0), lambda: L.expert_topk(p, 9),
        lambda: L.expert_topk(p[0], 2), lambda: L.expert_topk(p, 2, floor=math.nan),
        lambda: L.expert_topk(torch.rand(2, 1025, device=dev), 2), lambda: L.expert_topk(torch.rand(2, 100, device=dev), 65),
        lambda: L.expert_topk(torch.rand(2, 0, device=dev), 1),
        lambda: L.expert_sort(ids.long(), 3), lambda: L.expert_sort(ids, 0), lambda: L.expert_sort(ids, 1025),
        lambda: L.expert_sort(ids[0], 3), lambda: L.expert_sort(ids.t(), 3),
        lambda: L.expert_sort(torch.zeros(2, 65, dtype=torch.int32, device=dev), 3),
        lambda: L.expert_dispatch(x[:3], plan), lambda: L.expert_dispatch(x.double(), plan),
        lambda: L.expert_dispatch(x, L.ExpertPlan(4, plan.offsets, plan.order, plan.place)),
        lambda: L.expert_dispatch(x, L.ExpertPlan(3, plan.offsets, plan.order[:3], plan.place)),
        lambda: L.expert_dispatch(x, L.ExpertPlan(3, plan.offsets.cpu(), plan.order, plan.place)),
        lambda: L.expert_dispatch_vjp(xs[:, ::2], plan),
        lambda: L.expert_linear(xs, wt[:, :, :8], plan), lambda: L.expert_linear(xs, wt[:2], plan),
        lambda: L.expert_linear(xs, wt.half(), plan), lambda: L.expert_linear(xs, wt, plan, activation="tanh"),
        lambda: L.expert_linear(xs, wt, plan, bias=torch.zeros(3, 4, device=dev)),
        lambda: L.expert_linear(xs[:7], wt, plan), lambda: L.expert_linear(xs, wt[0], plan),
        lambda: L.expert_combine(xs, w[:3], plan), lambda: L.expert_combine(xs, w.half(), plan),
        lambda: L.expert_combine(xs, w, plan, residual=x[:, :8]), lambda: L.expert_combine(xs[:6], w, plan),
        lambda: L.expert_combine(xs, w, plan, residual=x.half()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(f"call {i} was not refused")
    for f in (lambda: L.expert_topk([1.0], 1), lambda: L.expert_dispatch(x, None),
              lambda: L.expert_linear(xs, None, plan), lambda: L.expert_combine(xs, [1.0], plan)):
        with pytest.raises(TypeError):
            f()


def test_only_what_requires_a_gradient_gets_one():
    T, m, E, K, F = 20, 2, 4, 16, 24
    plan, o, order, place = make_plan(some_ids(T, m, E, 1), E)
    g = gen(2)
    xs = torch.randn(T * m, K, generator=g).cuda()
    wt, b = torch.randn(E, F, K, generator=g).cuda(), torch.randn(E, F, generator=g).cuda()
    dy = torch.randn(T * m, F, generator=g).cuda()
    _, z = L.expert_linear_forward(xs, wt, plan, bias=b, activation="silu")
    want = L.expert_linear_vjp(xs, wt, plan, z, dy, activation="silu")
    for i in range(3):
        leaves = [t.detach().requires_grad_(i == j) for j, t in enumerate((xs, wt, b))]
        y = L.expert_linear(leaves[0], leaves[1], plan, bias=leaves[2], activation="silu")
        y.backward(dy)
        for j, t in enumerate(leaves):
            assert (t.grad is None) == (i != j)
        assert torch.equal(leaves[i].grad, want[i])
        alone = L.expert_linear_vjp(xs, wt, plan, z, dy, activation="silu", want=[i == j for j in range(3)])
        assert [t is None for t in alone] == [i != j for j in range(3)]
    x = torch.randn(T, F, generator=g).cuda()
    w = torch.rand(T, m, generator=g).cuda()
    both = L.expert_combine_vjp(dy, w, plan, x)
    for i in range(3):
        ys, wd, res = (t.detach().requires_grad_(i == j) for j, t in enumerate((dy, w, torch.zeros_like(x))))
        L.expert_combine(ys, wd, plan, residual=res).backward(x)
        for j, t in enumerate((ys, wd, res)):
            assert (t.grad is None) == (i != j)
            if i == j:
                assert torch.equal(t.grad, x if j == 2 else both[j])


def test_second_derivatives_are_refused():
    plan, *_ = make_plan(some_ids(6, 2, 3, 1), 3)
    x = torch.randn(6, 8, device="cuda", requires_grad=True)
    y = L.expert_dispatch(x, plan)
    with pytest.raises(RuntimeError, match="twice"):
        torch.autograd.grad(y.sum(), x, create_graph=True)


def test_a_plan_from_elsewhere_stays_in_bounds():
    """Places and offsets outside the pairs are empty slots and clamped ends."""
    T, m, E, D = 6, 2, 3, 32
    place = torch.tensor([[0, 99], [-5, 3], [2 ** 31 - 1, 1], [12, 2], [-1, -1], [4, 11]], dtype=torch.int32).cuda()
    offsets = torch.tensor([0, 3, 2 ** 31 - 1, 5], dtype=torch.int32).cuda()
    plan = L.ExpertPlan(E, offsets, torch.zeros(T * m, dtype=torch.int32).cuda(), place)
    x = torch.randn(T, D, generator=gen(1)).cuda()
    out = L.expert_combine(torch.ones(T * m, D).cuda(), torch.ones(T, m).cuda(), plan)
    ok = ((place >= 0) & (place < T * m)).sum(1).float().cpu()
    assert torch.equal(out.cpu(), ok[:, None].expand(T, D))
    assert L.expert_dispatch(x, plan).shape == (T * m, D)
    assert L.expert_linear(torch.ones(T * m, D).cuda(), torch.ones(E, 8, D).cuda(), plan).shape == (T * m, 8)


def block(x, gates, weights, m, E):
    ids, w = L.expert_topk(gates, m, normalize=True)
    plan = L.expert_sort(ids, E)
    w1, b1, w2 = weights
    h = L.expert_linear(L.expert_dispatch(x, plan), w1, plan, bias=b1, activation="silu")
    return L.expert_combine(L.expert_linear(h, w2, plan), w, plan, residual=x)


def block_inputs(T, E, K, F, dtype, seed=0):
    g = gen(seed)
    return (torch.randn(T, K, generator=g).to(dtype).cuda(), torch.rand(T, E, generator=g).cuda(),
            [(torch.randn(E, F, K, generator=g) * K ** -0.5).to(dtype).cuda(),
             torch.randn(E, F, generator=g).to(dtype).cuda(),
             (torch.randn(E, K, F, generator=g) * F ** -0.5).to(dtype).cuda()])


@pytest.mark.parametrize("T", [3, 300])
def test_on_another_stream_and_twice_the_same(T):
    x, gates, weights = block_inputs(T, 8, 128, 256, torch.bfloat16)
    want = block(x, gates, weights, 2, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [block(x, gates, weights, 2, 8) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for y in got:
        assert torch.equal(y, want)


@pytest.mark.parametrize("T", [4, 9000])
def test_graph_replays_follow_new_inputs(T):
    """Captured once, replayed with other gates and rows: the plan is made
    again inside the graph.  Every replay against the eager call."""
    E, m = 8, 2
    x, gates, weights = block_inputs(T, E, 64, 128, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            block(x, gates, weights, m, E)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x, gates, weights, m, E)
    for i in range(4):
        x1, g1, _ = block_inputs(T, E, 64, 128, torch.bfloat16, seed=10 + i)
        x.copy_(x1)
        gates.copy_(g1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, block(x, gates, weights, m, E)), i


@pytest.mark.slow
def test_rows_past_2_to_the_31_elements():
    """Offsets beyond 32 bits in dispatch, combine and the products."""
    D, T, E = 8192, 270_000, 2  # 2.2e9 elements
    ids = torch.zeros(T, 1, dtype=torch.int32)
    ids[::2] = 1
    plan = L.expert_sort(ids.cuda(), E)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    mark = torch.arange(T, device="cuda")
    x[:, 0] = (mark % 251).to(torch.bfloat16)
    x[:, D - 1] = (mark % 241).to(torch.bfloat16)
    xs = L.expert_dispatch(x, plan)
    token = plan.order.long()
    assert torch.equal(xs[:, 0], x[token, 0]) and torch.equal(xs[:, D - 1], x[token, D - 1])
    w = torch.full((T, 1), 2.0, device="cuda")
    out = L.expert_combine(xs, w, plan)
    assert torch.equal(out[:, 0], 2 * x[:, 0]) and torch.equal(out[:, D - 1], 2 * x[:, D - 1])
    del out
    # one output column per expert: the sum of a row's two marks, times e + 1
    weight = torch.zeros(E, 8, D, dtype=torch.bfloat16, device="cuda")
    weight[:, 3, 0] = weight[:, 3, D - 1] = torch.tensor([1.0, 2.0], device="cuda").to(torch.bfloat16)
    y = L.expert_linear(xs, weight, plan)
    ref = (xs[:, 0].float() + xs[:, D - 1].float()) * (ids.cuda().float()[token] + 1)[:, 0]
    assert torch.equal(y[:, 3], ref.to(torch.bfloat16))
    del y
    # and back: dx of a wide row
    dxs, dw, _ = L.expert_linear_vjp(xs, weight, plan, None, torch.ones(T, 8, dtype=torch.bfloat16, device="cuda"),
                                     want=(True, True, False))
    e1 = (ids.cuda()[token, 0] + 1).to(torch.bfloat16)
    assert torch.equal(dxs[:, 0], e1) and torch.equal(dxs[:, D - 1], e1)
    assert not dxs[:, 1:D - 1].any()
    for e in range(E):
        part = xs[int(plan.offsets[e]):int(plan.offsets[e + 1]), 0].double().sum()
        assert abs(float(dw[e, 5, 0]) - float(part)) <= 2.0 ** -8 * float(part) + T * R.EPS * float(part)
