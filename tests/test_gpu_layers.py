"""The norm, the loss and the experts' products in 8 bits against their
definitions in float64, forward and backward, at the sizes, targets, values and
alignments where they can go wrong.  Tolerances are the kernels' worst-case
rounding (layer_reference)."""
import math

import pytest
import torch

import expert_reference as X
import layer_reference as R

pytestmark = pytest.mark.gpu

L = pytest.importorskip("differentiable_exact_budget_amd")

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def put(*tensors):
    return [None if t is None else t.cuda() for t in tensors]


# ---- layer norm ------------------------------------------------------------------

def norm_case(T, D, dtype, wtype, affine=(True, True), seed=0):
    g = gen(seed + T + D)
    size = torch.exp(torch.randn(T, 1, generator=g))
    x = ((torch.randn(T, D, generator=g) + 0.5) * size).to(dtype)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(wtype) if affine[0] else None
    b = (0.3 * torch.randn(D, generator=g)).to(wtype) if affine[1] else None
    return x, w, b, torch.randn(T, D, generator=g).to(dtype)


def check_norm(x, w, b, dy, eps=1e-5, on="cpu"):
    leaves = [None if t is None else t.cuda().requires_grad_(True) for t in (x, w, b)]
    y = L.layer_norm(*leaves, eps=eps)
    ref = R.norm(*(None if t is None else t.to(on) for t in (x, w, b)), eps, dy.to(on))
    X.check(y, *ref["y"], "y")
    y1, mean, rstd = L.layer_norm_forward(*put(x, w, b), eps=eps)
    assert torch.equal(y1, y)
    X.check(mean, *ref["mean"], "mean")
    X.check(rstd, *ref["rstd"], "rstd")
    with torch.no_grad():
        assert torch.equal(L.layer_norm(*leaves, eps=eps), y)
    y.backward(dy.cuda())
    for name, t in zip(("dx", "dw", "db"), leaves):
        if t is not None:
            X.check(t.grad, *ref[name], name)


@pytest.mark.parametrize("T,D", [(1, 1), (1, 2), (3, 7), (5, 64), (4, 129), (9, 511), (7, 512), (6, 1000), (5, 1023),
                                 (3, 2047), (70, 2048), (33, 2049), (11, 4095), (5, 4096), (3, 8191), (4, 8193),
                                 (3, 16384)])
@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm(T, D, dtype):
    check_norm(*norm_case(T, D, dtype, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,D", [(3000, 64), (5, 333), (2500, 1024)])
def test_layer_norm_of_16_bit_rows_with_float32_weights(dtype, T, D):
    check_norm(*norm_case(T, D, dtype, torch.float32))


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_of_rows_that_registers_do_not_hold(dtype):
    check_norm(*norm_case(5, 40001, dtype, dtype))
    check_norm(*norm_case(70, 16392, dtype, torch.float32))


@pytest.mark.parametrize("affine", [(False, False), (True, False), (False, True)])
def test_layer_norm_without_weight_or_bias(affine):
    check_norm(*norm_case(40, 300, torch.bfloat16, torch.float32, affine))
    check_norm(*norm_case(6, 20000, torch.float32, torch.float32, affine))


def test_layer_norm_of_constant_and_offset_rows():
    """A constant row has the variance 0 (y is the bias); a row far from 0
    keeps the accuracy of values about the mean."""
    x = torch.full((3, 200), 7.5)
    w, b = torch.rand(200) + 0.5, torch.randn(200)
    assert torch.equal(L.layer_norm(*put(x, w, b)).cpu(), b.expand(3, 200))
    for D in (37, 3000, 30000):  # a value whose sums round
        assert torch.equal(L.layer_norm(torch.full((2, D), 7.3).cuda()).cpu(), torch.zeros(2, D))
    x = 1000.0 + torch.randn(6, 777, generator=gen(1))
    check_norm(x, w := torch.rand(777) + 0.5, torch.randn(777), torch.randn(6, 777))
    check_norm(x, w, None, torch.randn(6, 777), eps=0.0)


def test_layer_norm_of_no_rows_and_other_shapes():
    w, b = torch.rand(16, device="cuda", requires_grad=True), torch.rand(16, device="cuda", requires_grad=True)
    x = torch.empty(0, 16, device="cuda", requires_grad=True)
    y = L.layer_norm(x, w, b)
    y.sum().backward()
    assert y.shape == x.shape and torch.equal(w.grad, torch.zeros_like(w)) and torch.equal(b.grad, torch.zeros_like(b))
    x = torch.randn(2, 3, 16, device="cuda")
    flat = L.layer_norm(x.reshape(6, 16), w, b)
    assert torch.equal(L.layer_norm(x, w, b), flat.reshape(2, 3, 16))
    assert torch.equal(L.layer_norm(x[1, 2], w, b), flat[5])
    _, mean, rstd = L.layer_norm_forward(x, w, b)
    assert mean.shape == rstd.shape == (2, 3)


def test_layer_norm_of_values_that_are_not_finite_stays_in_its_row():
    x, w, b, _ = norm_case(6, 300, torch.float32, torch.float32)
    want = L.layer_norm(*put(x, w, b))
    x[1, 5], x[3, 0], x[4, 299] = math.inf, math.nan, -math.inf
    got = L.layer_norm(*put(x, w, b))
    for r in range(6):
        assert torch.equal(got[r], want[r]) if r in (0, 2, 5) else got[r].isnan().all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [3, 300, 5000, 20000])
def test_layer_norm_of_variances_past_float32(D, dtype):
    """Squares of 1e24 are infinite, and so is the variance: the result is the bias, the gradient 0."""
    x, w, b, dy = norm_case(4, D, dtype, dtype)
    want = L.layer_norm(*put(x, w, b))
    x[1], x[3] = torch.randn(2, D, generator=gen(2)).sign() * 1e24 + torch.randn(2, D, generator=gen(4)) * 1e23
    y, mean, rstd = L.layer_norm_forward(*put(x, w, b))
    dx, _, _ = L.layer_norm_vjp(*put(x, w), mean, rstd, dy.cuda())
    for r in range(4):
        if r in (0, 2):
            assert torch.equal(y[r], want[r])
        else:
            assert torch.equal(y[r].cpu(), b) and rstd[r] == 0 and not dx[r].any()


def test_layer_norm_of_other_strides_and_alignments():
    base = torch.randn(40, 130, generator=gen(3)).cuda()
    w, b = torch.rand(64, device="cuda"), torch.rand(64, device="cuda")
    for x in (base[:, 3:67], base[:, :128:2], base.t()[:64, :40].t(), base.reshape(-1)[1:1 + 64 * 40].reshape(40, 64)):
        x = x.detach().requires_grad_(True)
        plain = x.detach().clone().contiguous().requires_grad_(True)
        y, y0 = L.layer_norm(x, w, b), L.layer_norm(plain, w, b)
        assert torch.equal(y, y0)
        dy = torch.randn(64, 40, device="cuda").t()
        y.backward(dy)
        y0.backward(dy.contiguous())
        assert torch.equal(x.grad, plain.grad)
    for dtype in (torch.bfloat16, torch.float16):  # rows off 16 bytes
        x = base.to(dtype).reshape(-1)[1:1 + 64 * 40].reshape(40, 64)
        assert torch.equal(L.layer_norm(x, w, b), L.layer_norm(x.clone(), w, b))


def test_layer_norm_gradients_that_are_not_wanted_are_not_formed():
    x, w, b, dy = put(*norm_case(30, 100, torch.float32, torch.float32))
    y, mean, rstd = L.layer_norm_forward(x, w, b)
    want = L.layer_norm_vjp(x, w, mean, rstd, dy)
    for i in range(3):
        alone = L.layer_norm_vjp(x, w, mean, rstd, dy, want=[i == j for j in range(3)])
        assert torch.equal(alone[i], want[i]) and all(alone[j] is None for j in range(3) if j != i)
        leaves = [t.detach().requires_grad_(i == j) for j, t in enumerate((x, w, b))]
        L.layer_norm(*leaves).backward(dy)
        assert torch.equal(leaves[i].grad, want[i])
    bias = b.detach().requires_grad_(True)  # a bias without a weight
    L.layer_norm(x, None, bias).backward(dy)
    assert torch.equal(bias.grad, want[2])
    leaves = [t.detach().requires_grad_(True) for t in (x, w, b)]
    got = torch.autograd.grad(L.layer_norm(*leaves), leaves[1], dy)
    assert torch.equal(got[0], want[1])


# ---- the loss --------------------------------------------------------------------

def loss_case(T, V, D, dtype, bias=True, drop=0.2, scale=2.0, seed=0):
    g = gen(seed + T + V + D)
    x = torch.randn(T, D, generator=g).to(dtype)
    w = (torch.randn(V, D, generator=g) * scale * max(D, 1) ** -0.5).to(dtype)
    b = (0.5 * torch.randn(V, generator=g)).to(dtype) if bias else None
    target = torch.randint(V, (T,), generator=g)
    target[torch.rand(T, generator=g) < drop] = -100
    return x, w, b, target


def check_loss(x, w, b, target, reduction="mean", dloss=None, on="cpu"):
    leaves = [None if t is None else t.cuda().requires_grad_(True) for t in (x, w, b)]
    loss = L.linear_cross_entropy(leaves[0], leaves[1], target.cuda(), bias=leaves[2], reduction=reduction)
    if dloss is None:
        dloss = torch.rand(loss.shape, generator=gen(5)) + 0.5
        if x.dtype == torch.float16:
            dloss = dloss * 1024
    ref = R.loss(*(None if t is None else t.to(on) for t in (x, w, b, target)), reduction, dloss.to(on))
    X.check(loss, *ref["loss"], "loss")
    assert loss.dtype == torch.float32
    loss1, lse = L.linear_cross_entropy_forward(*put(x, w, target), bias=put(b)[0], reduction=reduction)
    assert torch.equal(loss1, loss)
    X.check(lse, *ref["lse"], "lse")
    with torch.no_grad():
        assert torch.equal(L.linear_cross_entropy(leaves[0], leaves[1], target.cuda(), bias=leaves[2],
                                                  reduction=reduction), loss)
    loss.backward(dloss.cuda())
    for name, t in zip(("dx", "dw", "db"), leaves):
        if t is not None:
            X.check(t.grad, *ref[name], name)
            assert t.grad.dtype == t.dtype
    return leaves


@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 2, 8), (2, 3, 5), (5, 17, 64), (7, 64, 40), (16, 129, 32), (33, 63, 72),
                                   (3, 1000, 257), (64, 128, 128), (65, 257, 96), (130, 255, 200), (200, 1001, 64),
                                   (17, 2050, 24), (300, 515, 136)])
@pytest.mark.parametrize("dtype", TYPES)
def test_loss(T, V, D, dtype):
    check_loss(*loss_case(T, V, D, dtype))


@pytest.mark.parametrize("T,V,D", [(1, 40000, 64), (4, 70001, 128), (3000, 700, 64), (1500, 3000, 320), (1024, 9000, 256)])
@pytest.mark.parametrize("dtype", TYPES)
def test_loss_of_many_rows_and_of_a_large_vocabulary(T, V, D, dtype):
    check_loss(*loss_case(T, V, D, dtype, bias=T % 2 == 0), on="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_loss_reductions_without_bias(dtype, reduction):
    check_loss(*loss_case(90, 300, 48, dtype, bias=False), reduction=reduction)
    check_loss(*loss_case(40, 120, 17, dtype, bias=False), reduction=reduction)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_loss_in_pieces_of_the_vocabulary(dtype):
    """Rows enough that a gradient's piece holds 256 or 128 columns."""
    T = (1 << 27) // 256 // 400 * 400 + 3 if dtype == torch.bfloat16 else (1 << 25) // 128 // 200 * 200 + 3
    check_loss(*loss_case(T, 700, 8, dtype, drop=0.9), on="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 33])
def test_loss_of_rows_without_a_target(dtype, D):
    """Targets outside [0, V) on either side; all rows of a call ignored; a
    row's logits may be anything then."""
    x, w, b, target = loss_case(50, 200, D, dtype, drop=0.0)
    target[3], target[10], target[20], target[21] = -1, 200, 2 ** 40, -2 ** 62
    check_loss(x, w, b, target)
    x[3] = math.nan
    x[10] = math.inf
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    L.linear_cross_entropy(leaves[0], leaves[1], target.cuda(), bias=leaves[2]).backward()
    assert leaves[0].grad[[3, 10, 20, 21]].abs().max() == 0
    assert leaves[0].grad.isfinite().all() and leaves[2].grad.isfinite().all()
    target[:] = -100
    x, w, b, _ = loss_case(50, 200, D, dtype)
    for reduction in ("none", "sum", "mean"):
        leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
        loss = L.linear_cross_entropy(leaves[0], leaves[1], target.cuda(), bias=leaves[2], reduction=reduction)
        assert loss.abs().max() == 0
        loss.sum().backward()
        assert all(t.grad.abs().max() == 0 for t in leaves)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 33])
def test_loss_of_masked_vocabularies(dtype, D):
    """A bias of -inf, or of the type's lowest value, takes entries out; a
    masked target has an infinite loss, a row with nothing left none at all."""
    x, w, b, target = loss_case(70, 500, D, dtype, drop=0.0)
    masked = torch.rand(500, generator=gen(2)) < 0.5
    masked[target] = False
    masked[256:384] = ~torch.isin(torch.arange(256, 384), target)  # nearly whole tiles
    b[masked] = -math.inf
    leaves = check_loss(x, w, b, target)
    assert leaves[1].grad[masked.cuda()].abs().max() == 0
    b[masked] = torch.finfo(dtype).min
    low = L.linear_cross_entropy(*put(x, w, target), bias=b.cuda(), reduction="none")
    b[masked] = -math.inf
    assert torch.equal(low, L.linear_cross_entropy(*put(x, w, target), bias=b.cuda(), reduction="none"))
    target[0] = int(masked.nonzero()[0])
    loss = L.linear_cross_entropy(*put(x, w, target), bias=b.cuda(), reduction="none").cpu()
    assert loss[0] == math.inf and torch.equal(loss[1:], low.cpu()[1:])
    b[:] = -math.inf
    assert L.linear_cross_entropy(*put(x, w, target), bias=b.cuda(), reduction="none").isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_loss_of_far_logits(dtype):
    """Logits in the hundreds: nothing overflows, and a sure row's loss is 0."""
    check_loss(*loss_case(40, 300, 64, dtype, scale=60.0))
    x = torch.zeros(3, 8)
    x[:, 0] = 1.0
    w = torch.zeros(10, 8)
    w[4, 0] = 200.0
    loss = L.linear_cross_entropy(*put(x.to(dtype), w.to(dtype)), torch.tensor([4, 4, 5]).cuda(), reduction="none")
    assert loss[:2].abs().max() == 0 and abs(float(loss[2]) - 200) < 1e-4


def test_loss_of_float16_keeps_small_gradients():
    """Gradients of rows' losses far below what float16 holds, and above."""
    x, w, b, target = loss_case(200, 600, 64, torch.float16)
    ref = None
    for scale in (2.0 ** -30, 1.0, 2.0 ** 20):
        leaves = [t.cuda() for t in (x, w, b)]
        _, lse = L.linear_cross_entropy_forward(leaves[0], leaves[1], target.cuda(), bias=leaves[2], reduction="none")
        # rows that bring every result into float16's range again
        dloss = torch.full((200,), scale, device="cuda")
        w2 = (w.float() / scale).clamp(-6e4, 6e4).half().cuda() if scale > 1 else leaves[1]
        dx, dw, db = L.linear_cross_entropy_vjp(leaves[0], leaves[1], target.cuda(), lse, dloss, bias=leaves[2],
                                                reduction="none", want=(True, True, True))
        r = R.loss(x, w, b, target, "none", dloss.cpu())
        for name, got in (("dx", dx), ("dw", dw), ("db", db)):
            value, tol = r[name]
            fits = value.abs() < 65000
            X.check(got.cpu()[fits], value[fits], tol[fits], f"{name} at {scale}")


def test_loss_of_no_rows_and_no_width_and_other_shapes():
    for dtype in TYPES:
        w, b = torch.rand(30, 16, device="cuda", dtype=dtype), torch.rand(30, device="cuda", dtype=dtype)
        x = torch.empty(0, 16, device="cuda", dtype=dtype)
        leaves = [t.requires_grad_(True) for t in (x, w, b)]
        for reduction in ("none", "sum", "mean"):
            loss = L.linear_cross_entropy(x, w, torch.empty(0, dtype=torch.int64, device="cuda"), bias=b,
                                          reduction=reduction)
            assert loss.numel() == (0 if reduction == "none" else 1) and loss.sum() == 0
            for t in leaves:
                t.grad = None
            loss.sum().backward()
            assert x.grad.shape == x.shape and w.grad.abs().max() == 0 and b.grad.abs().max() == 0
        empty = torch.empty(5, 0, device="cuda", dtype=dtype)
        target = torch.arange(5, device="cuda")
        loss = L.linear_cross_entropy(empty, torch.empty(30, 0, device="cuda", dtype=dtype), target, bias=b,
                                      reduction="none")
        X.check(loss, torch.logsumexp(b.detach().double().cpu(), 0) - b.detach().double().cpu()[:5],
                torch.full((5,), 1e-5, dtype=torch.float64), "loss")
    x, w, b, target = put(*loss_case(24, 50, 16, torch.float32))
    flat = L.linear_cross_entropy(x, w, target, bias=b, reduction="none")
    got = L.linear_cross_entropy(x.reshape(2, 3, 4, 16), w, target.reshape(2, 3, 4), bias=b, reduction="none")
    assert torch.equal(got, flat.reshape(2, 3, 4))
    assert torch.equal(L.linear_cross_entropy(x[5], w, target[5], bias=b, reduction="none"), flat[5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_loss_of_other_strides_and_alignments(dtype):
    x, w, b, target = put(*loss_case(40, 90, 64, dtype))
    want = [t.requires_grad_(True) for t in (x, w, b)]
    L.linear_cross_entropy(x, w, target, bias=b).backward()

    def off(t):  # the same values, one element off 16 bytes
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.detach().reshape(-1)
        return flat[1:].reshape(t.shape)

    def strided(t):
        wide = torch.empty(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device="cuda")
        wide[..., ::2] = t.detach()
        return wide[..., ::2]

    for change in (off, strided):
        got = [change(t).requires_grad_(True) for t in want]
        L.linear_cross_entropy(got[0], got[1], change(target), bias=got[2]).backward()
        ref = R.loss(x.detach().cpu(), w.detach().cpu(), b.detach().cpu(), target.cpu(), "mean", torch.ones(()))
        for name, t in zip(("dx", "dw", "db"), got):
            X.check(t.grad, *ref[name], name)


def test_loss_gradients_that_are_not_wanted_are_not_formed():
    for D in (64, 33):
        x, w, b, target = put(*loss_case(30, 100, D, torch.bfloat16))
        _, lse = L.linear_cross_entropy_forward(x, w, target, bias=b)
        one = torch.ones((), device="cuda")
        want = L.linear_cross_entropy_vjp(x, w, target, lse, one, bias=b, want=(True, True, True))
        for i in range(3):
            alone = L.linear_cross_entropy_vjp(x, w, target, lse, one, bias=b, want=[i == j for j in range(3)])
            assert torch.equal(alone[i], want[i]) and all(alone[j] is None for j in range(3) if j != i)
            leaves = [t.detach().requires_grad_(i == j) for j, t in enumerate((x, w, b))]
            L.linear_cross_entropy(leaves[0], leaves[1], target, bias=leaves[2]).backward()
            assert torch.equal(leaves[i].grad, want[i])


# ---- 8 bits ----------------------------------------------------------------------

@pytest.mark.parametrize("T,D", [(1, 1), (3, 127), (2, 128), (5, 129), (4, 300), (7, 1000), (3, 2048), (2, 2049), (9, 4111)])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize(T, D, dtype):
    g = gen(T + D)
    x = (torch.randn(T, D, generator=g) * torch.exp(3 * torch.randn(T, 1, generator=g))).to(dtype)
    x[0, ::3] = 0
    q, e = R.quantize(x)
    rows = L.expert_quantize(x.cuda())
    assert rows.shape == x.shape and rows.width == D
    assert torch.equal(rows.values.cpu().double(), q)
    assert torch.equal(rows.scales.view(torch.uint8).cpu().long(), e + 127)
    for out in TYPES:
        want = R.stands_for(q, e, D).to(out)
        assert torch.equal(L.expert_dequantize(rows, out).cpu(), want)
    # what 8 bits stand for stays (a block whose largest value was rounded down to
    # a border, 225 to 224, takes half the scale and twice the values)
    back = L.expert_dequantize(rows, torch.float32)
    assert torch.equal(L.expert_dequantize(L.expert_quantize(back), torch.float32), back)


def test_quantize_borders_and_unusual_values():
    """Powers of two and both sides of 448 2^e, ties, zeros of either sign, the
    smallest numbers, and what is not finite."""
    inf, nan = math.inf, math.nan
    row = lambda *v: torch.tensor(list(v) + [0.0] * (128 - len(v)))  # noqa: E731
    up = torch.nextafter(torch.tensor(448.0), torch.tensor(1e9)).item()
    x = torch.stack([
        row(448.0, 1.0, -2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10), row(up, 1.0, 2.0 ** -9), row(0.0, -0.0),
        row(1.0, 1.0625, 1.1875, -1.0625, 1.0624), row(2.0 ** 127 * 1.5, 2.0 ** 120), row(2.0 ** -126, -2.0 ** -127),
        row(2.0 ** -149), row(nan, 1.0, 2.0), row(inf, -inf, 3.0), row(nan), row(1.75 * 2.0 ** 100), row(1.76 * 2.0 ** 100),
    ])
    q, e = R.quantize(x)
    rows = L.expert_quantize(x.cuda())
    got = rows.values.cpu().double()
    assert torch.equal(got.isnan(), q.isnan())
    assert torch.equal(got.nan_to_num(), q.nan_to_num())
    assert torch.equal(torch.signbit(got[2]), torch.signbit(x[2]))
    assert torch.equal(rows.scales.view(torch.uint8).cpu().long(), e + 127)
    back = L.expert_dequantize(rows, torch.float32).cpu()
    want = R.stands_for(q, e, 128).float()
    assert torch.equal(back.nan_to_num(), want.nan_to_num()) and torch.equal(back.isnan(), want.isnan())
    rows.scales.view(torch.uint8)[1] = 255  # a scale of NaN
    assert L.expert_dequantize(rows).cpu()[1].isnan().all()


def test_quantize_of_nothing_and_other_shapes():
    for shape in ((0, 5), (4, 0), (2, 0, 7)):
        rows = L.expert_quantize(torch.empty(shape, device="cuda"))
        assert rows.shape == shape and L.expert_dequantize(rows).shape == shape
    x = torch.randn(2, 3, 200, device="cuda")
    rows, flat = L.expert_quantize(x), L.expert_quantize(x.reshape(6, 200))
    assert rows.values.shape == (2, 3, 256) and rows.scales.shape == (2, 3, 2)
    assert torch.equal(rows.values.view(torch.uint8).reshape(6, 256), flat.values.view(torch.uint8))
    assert torch.equal(L.expert_dequantize(rows, torch.float32).reshape(6, 200), L.expert_dequantize(flat, torch.float32))
    wide = torch.randn(6, 401, device="cuda")
    assert torch.equal(L.expert_quantize(wide[:, 1::2]).values.view(torch.uint8),
                       L.expert_quantize(wide[:, 1::2].clone()).values.view(torch.uint8))


def product8_case(T, m, E, K, F, dtype, bias=True, drop=0.2, idle=(), seed=0):
    g = gen(seed + T + K + F)
    score = torch.rand(T, E, generator=g)
    ids = score.topk(m, dim=1).indices.int()
    ids[torch.rand(T, m, generator=g) < drop] = -1
    for e in idle:
        ids[ids == e] = -1
    o, order, place = X.sort(ids, E)
    plan = L.ExpertPlan(E, *put(o, order, place))
    xs = torch.randn(T * m, K, generator=g) * torch.exp(torch.randn(T * m, 1, generator=g))
    w = torch.randn(E, F, K, generator=g) * max(K, 1) ** -0.5
    b = torch.randn(E, F, generator=g).to(dtype) if bias else None
    return plan, o, xs, w, b


def check_product8(plan, o, xs, w, b, act, dtype, on="cpu"):
    qx, qw = L.expert_quantize(xs.cuda()), L.expert_quantize(w.cuda())
    y = L.expert_linear_fp8(qx, qw, plan, bias=put(b)[0], activation=act, dtype=dtype)
    assert y.dtype == dtype
    sx, sw = (L.expert_dequantize(r, torch.float32).double().to(on) for r in (qx, qw))
    X.check(y, *R.linear8(sx, sw, None if b is None else b.to(on), o, act, dtype), "ys")
    return y


@pytest.mark.parametrize("T,m,E,K,F", [(1, 1, 1, 1, 1), (1, 2, 4, 128, 64), (3, 1, 2, 130, 5), (4, 4, 64, 256, 96),
                                       (33, 2, 3, 65, 63), (100, 2, 7, 257, 130), (300, 2, 5, 512, 264),
                                       (64, 2, 4, 2047, 200), (16, 4, 16, 1024, 512), (20, 2, 3, 2200, 48),
                                       (500, 1, 2, 4300, 72)])
@pytest.mark.parametrize("dtype", TYPES)
def test_products_in_8_bits(T, m, E, K, F, dtype):
    check_product8(*product8_case(T, m, E, K, F, dtype), "silu", dtype)


@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
@pytest.mark.parametrize("T,m,E,K,F", [(70, 2, 4, 384, 200), (9, 1, 3, 100, 31)])
def test_products_in_8_bits_other_activations(act, T, m, E, K, F):
    for dtype in TYPES:
        check_product8(*product8_case(T, m, E, K, F, dtype, bias=act == "relu"), act, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,m,E,K,F", [(2000, 2, 3, 1024, 1000), (5000, 2, 8, 256, 2048), (4100, 2, 4, 2304, 1032),
                                       (3000, 2, 5, 300, 777)])
def test_products_in_8_bits_of_many_rows(dtype, T, m, E, K, F):
    check_product8(*product8_case(T, m, E, K, F, dtype, idle=(1,)), "silu", dtype, on="cuda")


def test_products_in_8_bits_leave_idle_experts_and_unused_rows_alone():
    """Weights of experts without rows, and rows past the used ones, may hold
    NaN; unused rows of the result are zeros."""
    plan, o, xs, w, b = product8_case(300, 2, 6, 256, 136, torch.bfloat16, idle=(0, 4))
    used = int(o[-1])
    want = check_product8(plan, o, xs, w, b, "silu", torch.bfloat16)
    xs[used:] = math.nan
    w[0] = w[4] = math.nan
    b[0] = b[4] = math.nan
    qx, qw = L.expert_quantize(xs.cuda()), L.expert_quantize(w.cuda())
    qw.scales.view(torch.uint8)[4] = 255
    qx.scales.view(torch.uint8)[used:] = 255
    y = L.expert_linear_fp8(qx, qw, plan, bias=b.cuda(), activation="silu")
    assert torch.equal(y, want) and used < 600 and y[used:].abs().max() == 0


def test_products_in_8_bits_of_nothing():
    plan, o, xs, w, b = product8_case(4, 2, 3, 256, 16, torch.float32)
    q, qw = L.expert_quantize(xs.cuda()), L.expert_quantize(w.cuda())
    none = L.expert_sort(torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), 3)
    assert L.expert_linear_fp8(q, qw, none, bias=b.cuda(), dtype=torch.float32).abs().max() == 0
    empty = L.expert_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    assert L.expert_linear_fp8(L.expert_quantize(xs[:0].cuda()), qw, empty).shape == (0, 16)
    assert L.expert_linear_fp8(q, L.expert_quantize(w[:, :0].cuda()), plan).shape == (8, 0)
    y = L.expert_linear_fp8(L.expert_quantize(xs[:, :0].cuda()), L.expert_quantize(w[:, :, :0].cuda()), plan,
                            bias=b.cuda(), dtype=torch.float32)
    for e in range(3):
        assert torch.equal(y[int(o[e]):int(o[e + 1])].cpu(), b[e].expand(int(o[e + 1] - o[e]), 16))


def test_products_in_8_bits_of_values_that_are_not_finite_stay_in_their_row():
    plan, o, xs, w, b = product8_case(40, 2, 3, 384, 72, torch.float32, drop=0.0)
    want = check_product8(plan, o, xs, w, b, "none", torch.float32)
    xs[5, 200] = math.nan
    xs[17, 0] = math.inf
    got = L.expert_linear_fp8(*(L.expert_quantize(t.cuda()) for t in (xs, w)), plan, bias=b.cuda(), dtype=torch.float32)
    rest = [r for r in range(80) if r not in (5, 17)]
    assert torch.equal(got[rest], want[rest]) and got[[5, 17]].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_products_in_8_bits_of_the_least_and_of_missing_scales(dtype):
    """Scales from 2^-127 on, whose products come back into range, and scales of
    NaN, which make their row (of the rows) or column (of the weights) NaN."""
    g = gen(8)
    K, F, P = 256, 40, 70
    xs = torch.randn(P, K, generator=g) * torch.exp2(torch.randint(-126, -100, (P, 1), generator=g).float())
    xs[:8] = torch.randn(8, K, generator=g) * 2.0 ** -128
    w = torch.randn(1, F, K, generator=g) * 2.0 ** 110
    plan = L.expert_sort(torch.zeros(P, 1, dtype=torch.int32, device="cuda"), 1)
    o = torch.tensor([0, P])
    want = check_product8(plan, o, xs, w, None, "none", dtype)
    assert want.abs().max() > 0
    qx, qw = L.expert_quantize(xs.cuda()), L.expert_quantize(w.cuda())
    assert int(qx.scales.view(torch.uint8).min()) == 0
    qx.scales.view(torch.uint8)[5, 1] = 255
    qw.scales.view(torch.uint8)[0, 33, 0] = 255
    got = L.expert_linear_fp8(qx, qw, plan, dtype=dtype)
    bad = torch.zeros(P, F, dtype=torch.bool)
    bad[5], bad[:, 33] = True, True
    assert torch.equal(got.isnan().cpu(), bad) and torch.equal(got.cpu()[~bad], want.cpu()[~bad])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_in_8_bits_by_a_plan_from_elsewhere_stay_in_bounds(dtype):
    """Offsets that run back or past the rows: rows may be wrong, and nothing
    outside the arrays is read or written (the results have guards around them)."""
    P, E, K, F = 600, 6, 256, 136
    g = gen(12)
    qx = L.expert_quantize(torch.randn(P, K, generator=g).cuda())
    qw = L.expert_quantize(torch.randn(E, F, K, generator=g).cuda())
    for off in ([0, P] * 3 + [0], [0, 900, 100, -5, 2 ** 31 - 1, 700, 650], [P] * 7, [-(2 ** 31)] * 7):
        plan = L.ExpertPlan(E, torch.tensor(off, dtype=torch.int32).cuda(), torch.zeros(P, dtype=torch.int32).cuda(),
                            torch.zeros(P // 2, 2, dtype=torch.int32).cuda())
        y = L.expert_linear_fp8(qx, qw, plan, dtype=dtype)
        assert y.shape == (P, F)
    torch.cuda.synchronize()


# ---- refusals --------------------------------------------------------------------

def test_refusals():
    dev = "cuda"
    x, w = torch.rand(6, 128, device=dev), torch.rand(10, 128, device=dev)
    t = torch.zeros(6, dtype=torch.int64, device=dev)
    plan = L.expert_sort(torch.zeros(6, 1, dtype=torch.int32, device=dev), 2)
    q, qw = L.expert_quantize(x), L.expert_quantize(torch.rand(2, 16, 128, device=dev))
    v8, s8 = q.values, q.scales
    for f in (
        lambda: L.layer_norm(x.double()), lambda: L.layer_norm(x[:, :0]), lambda: L.layer_norm(x, w[0].half()),
        lambda: L.layer_norm(x, w[0, :64]), lambda: L.layer_norm(x, w[0], w[0].bfloat16()), lambda: L.layer_norm(x, w[0].cpu()),
        lambda: L.layer_norm(x, eps=-1.0), lambda: L.layer_norm(x, eps=math.nan), lambda: L.layer_norm(x.sum()),
        lambda: L.layer_norm_vjp(x, None, t.float(), t.float(), x[:, :64]),
        lambda: L.layer_norm_vjp(x, None, t.float()[:5], t.float(), x),
        lambda: L.linear_cross_entropy(x, w.half(), t), lambda: L.linear_cross_entropy(x, w[:, :64], t),
        lambda: L.linear_cross_entropy(x, w[0], t), lambda: L.linear_cross_entropy(x, w[:0], t),
        lambda: L.linear_cross_entropy(x, w, t.int()), lambda: L.linear_cross_entropy(x, w, t[:5]),
        lambda: L.linear_cross_entropy(x, w, t.cpu()), lambda: L.linear_cross_entropy(x, w, t, bias=w[0]),
        lambda: L.linear_cross_entropy(x, w, t, bias=w[:, 0].half()), lambda: L.linear_cross_entropy(x, w, t, reduction="max"),
        lambda: L.linear_cross_entropy(x.double(), w.double(), t),
        lambda: L.linear_cross_entropy_vjp(x, w, t, t.float(), t.float()),
        lambda: L.linear_cross_entropy_vjp(x, w, t, t.float()[:5], t.float().sum()),
        lambda: L.expert_quantize(x.double()), lambda: L.expert_quantize(x.sum()),
        lambda: L.expert_dequantize(q, torch.float64),
        lambda: L.expert_dequantize(L.ScaledRows(v8, s8, 129)), lambda: L.expert_dequantize(L.ScaledRows(v8, s8, -1)),
        lambda: L.expert_dequantize(L.ScaledRows(v8.view(torch.uint8), s8, 128)),
        lambda: L.expert_dequantize(L.ScaledRows(v8, s8.view(torch.uint8), 128)),
        lambda: L.expert_dequantize(L.ScaledRows(v8, s8[:5], 128)), lambda: L.expert_dequantize(L.ScaledRows(v8[:, :64], s8, 64)),
        lambda: L.expert_dequantize(L.ScaledRows(v8.view(torch.uint8).reshape(-1)[1:129].view(torch.float8_e4m3fn), s8[0], 128)),
        lambda: L.expert_linear_fp8(q, L.expert_quantize(torch.rand(3, 16, 128, device=dev)), plan),
        lambda: L.expert_linear_fp8(q, L.expert_quantize(torch.rand(2, 16, 100, device=dev)), plan),
        lambda: L.expert_linear_fp8(L.expert_quantize(x[:5]), qw, plan),
        lambda: L.expert_linear_fp8(q, q, plan), lambda: L.expert_linear_fp8(q, qw, plan, activation="tanh"),
        lambda: L.expert_linear_fp8(q, qw, plan, bias=torch.zeros(2, 16, device=dev)),
        lambda: L.expert_linear_fp8(q, qw, plan, bias=torch.zeros(2, 15, device=dev, dtype=torch.bfloat16)),
        lambda: L.expert_linear_fp8(q, qw, plan, dtype=torch.float64),
    ):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: L.expert_linear_fp8(x, qw, plan), lambda: L.expert_linear_fp8(q, qw, None),
              lambda: L.expert_dequantize(q, "bfloat16"), lambda: L.linear_cross_entropy(x, w, [0] * 6)):
        with pytest.raises(TypeError):
            f()
    bias = torch.zeros(2, 16, device=dev, dtype=torch.bfloat16, requires_grad=True)
    kept = L.ScaledRows(q.values.detach().requires_grad_(True), q.scales, 128)
    for f in (lambda: L.expert_quantize(x.detach().requires_grad_(True)), lambda: L.expert_linear_fp8(q, qw, plan, bias=bias),
              lambda: L.expert_dequantize(kept), lambda: L.expert_linear_fp8(kept, qw, plan)):
        with pytest.raises(RuntimeError, match="no gradient"):
            f()
        with torch.no_grad():
            f()


def calls():
    x, w, b, _ = put(*norm_case(6, 40, torch.float32, torch.float32))
    lx, lw, lb, t = put(*loss_case(6, 30, 40, torch.float32))
    return {"layer_norm": (lambda x, w, b: L.layer_norm(x, w, b), (x, w, b)),
            "linear_cross_entropy": (lambda x, w, b: L.linear_cross_entropy(x, w, t, bias=b), (lx, lw, lb))}


@pytest.mark.parametrize("name", ["layer_norm", "linear_cross_entropy"])
def test_what_has_no_derivative_is_refused(name):
    """Forward-mode tangents, second derivatives, and traces."""
    call, inputs = calls()[name]
    fw = torch.autograd.forward_ad
    with fw.dual_level():
        for i in range(3):
            dual = [fw.make_dual(t, torch.ones_like(t)) if i == j else t for j, t in enumerate(inputs)]
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(*dual)
    leaves = [t.detach().requires_grad_(True) for t in inputs]
    with pytest.raises(RuntimeError, match="twice"):
        torch.autograd.grad(call(*leaves).sum(), leaves, create_graph=True)
    for grad in (False, True):
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(call, tuple(t.detach().requires_grad_(grad) for t in inputs), check_trace=False)


# ---- differences, streams, graphs, a model of them ---------------------------------

def test_gradients_against_differences():
    """The float32 gradients along random directions against central
    differences of the same calls in steps that float32 resolves: the loss is
    about 1, its evaluations are off by some 1e-6, the differences by 1e-6 / h and
    by h^2 of a third derivative that is about 1."""
    g = gen(9)
    x, w, b, _ = norm_case(20, 50, torch.float32, torch.float32)
    _, v, vb, target = loss_case(20, 70, 50, torch.float32)
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b, v, vb)]

    def value(x, w, b, v, vb):
        return L.linear_cross_entropy(L.layer_norm(x, w, b), v, target.cuda(), bias=vb)

    grads = torch.autograd.grad(value(*leaves), leaves)
    h = 1e-2
    for i, t in enumerate(leaves):
        way = torch.randn(t.shape, generator=g).cuda()
        way = way / way.norm()
        with torch.no_grad():
            ends = [value(*(u + s * h * way if i == j else u for j, u in enumerate(leaves))) for s in (1, -1)]
        slope = float((ends[0].double() - ends[1].double()) / (2 * h))
        assert abs(slope - float((grads[i].double() * way.double()).sum())) < 5e-4, i


def model(x, p, plan_of, fp8=None):
    """norm, gates, experts, combine and the loss, as they are used together."""
    h = L.layer_norm(x, p["nw"], p["nb"])
    plan, gates = plan_of(h)
    hs = L.expert_dispatch(h, plan)
    if fp8 is None:
        a = L.expert_linear(hs, p["w1"], plan, bias=p["b1"], activation="silu")
        ys = L.expert_linear(a, p["w2"], plan)
    else:
        a = L.expert_linear_fp8(L.expert_quantize(hs), fp8[0], plan, bias=p["b1"], activation="silu", dtype=x.dtype)
        ys = L.expert_linear_fp8(L.expert_quantize(a), fp8[1], plan, dtype=x.dtype)
    out = L.expert_combine(ys, gates, plan, residual=x)
    return L.linear_cross_entropy(L.layer_norm(out, p["ow"], p["ob"]), p["v"], p["target"], bias=p["vb"])


def model_inputs(T, dtype, seed=0, D=64, F=128, E=4, V=500):
    g = gen(100 + seed)
    r = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(dtype).cuda()  # noqa: E731
    p = {"nw": 1 + r(D, scale=0.1), "nb": r(D, scale=0.1), "w1": r(E, F, D, scale=D ** -0.5), "b1": r(E, F, scale=0.1),
         "w2": r(E, D, F, scale=F ** -0.5), "ow": 1 + r(D, scale=0.1), "ob": r(D, scale=0.1),
         "v": r(V, D, scale=2 * D ** -0.5), "vb": r(V, scale=0.1)}
    router = torch.randn(E, D, generator=g).cuda()
    p["target"] = torch.randint(-20, V, (T,), generator=g).cuda()
    x = r(T, D)

    def plan_of(h):
        gates = L.soft_topk_rows(h.float() @ router.t(), 2.0, 0.3)
        ids, w = L.expert_topk(gates, 2)
        return L.expert_sort(ids, E), w

    return x, p, plan_of


@pytest.mark.parametrize("dtype", TYPES)
def test_a_model_of_them(dtype):
    """Training: the gradients of norm, router, experts and loss together
    against the same formulas in float64 with the same choice of experts.  Each
    of about ten roundings to the rows' type adds u / sqrt(3) in the 2-norm, a
    gradient passes all of them, and 12 of them are allowed.  Serving: the experts
    in 8 bits, off by e4m3's 2^-4 / sqrt(3) of each product's two operands."""
    T, E = 300, 4
    x, p, plan_of = model_inputs(T, dtype)
    scale = 256.0 if dtype == torch.float16 else 1.0
    leaves = {k: t.detach().requires_grad_(t.is_floating_point()) for k, t in p.items()}
    xl = x.detach().requires_grad_(True)
    kept = {}

    def keep(h):
        kept["plan"], kept["w"] = plan_of(h)
        return kept["plan"], kept["w"].detach()  # the router's own gradient has tests of its own

    loss = model(xl, leaves, keep)
    names = [k for k in p if k != "target"]
    grads = torch.autograd.grad(loss * scale, [xl] + [leaves[k] for k in names])

    ref = {k: t.detach().double().requires_grad_(True) for k, t in p.items() if k != "target"}
    xr = x.double().requires_grad_(True)
    h = torch.nn.functional.layer_norm(xr, xr.shape[-1:], ref["nw"], ref["nb"])
    place, order = kept["plan"].place.long(), kept["plan"].order
    off = kept["plan"].offsets.tolist()
    out = xr
    token = (order.clamp(min=0) // 2).long()
    flat = kept["w"].double().reshape(-1)[order.clamp(min=0).long()]
    for e in range(E):
        r = slice(off[e], off[e + 1])
        a = torch.nn.functional.silu(h[token[r]] @ ref["w1"][e].t() + ref["b1"][e])
        out = out.index_add(0, token[r], (a @ ref["w2"][e].t()) * flat[r, None])
    z = torch.nn.functional.layer_norm(out, out.shape[-1:], ref["ow"], ref["ob"]) @ ref["v"].t() + ref["vb"]
    target = torch.where(p["target"] < 0, -100, p["target"])
    want = torch.nn.functional.cross_entropy(z, target)
    wants = torch.autograd.grad(want * scale, [xr] + [ref[k] for k in names])
    u = R.U[dtype] / math.sqrt(3)
    assert abs(float(loss.detach()) - float(want.detach())) < 12 * u * abs(float(want.detach())) + 1e-5
    for name, got, w in zip(["x"] + names, grads, wants):
        rel = float((got.double() - w).norm() / w.norm())
        assert rel < 12 * u + 2e-5, (name, rel)
    with torch.no_grad():
        eight = model(x, p, lambda h: (kept["plan"], kept["w"]), [L.expert_quantize(p[k]) for k in ("w1", "w2")])
    # the experts' part of the rows is off by 4 roundings of 2^-4 / sqrt(3), 0.07
    # of it, and the logits and the loss by less than that share of the loss
    assert abs(float(eight) - float(loss)) < 0.07 * float(loss)


@pytest.mark.parametrize("T", [3, 400])
def test_on_another_stream_and_twice_the_same(T):
    x, p, plan_of = model_inputs(T, torch.bfloat16)

    def step():
        leaves = [p[k].detach().requires_grad_(True) for k in ("nw", "v", "vb")]
        q = dict(p, nw=leaves[0], v=leaves[1], vb=leaves[2])
        loss = model(x, q, plan_of)
        return [loss.detach(), *torch.autograd.grad(loss, leaves)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [step() for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_graph_replays_follow_new_inputs(T, dtype):
    """A training step of the norm and the loss, and a serving step in 8 bits,
    captured once and replayed with other rows and targets; every replay against
    the eager calls, which run between them."""
    x, p, plan_of = model_inputs(T, dtype)
    q1, q2 = L.expert_quantize(p["w1"]), L.expert_quantize(p["w2"])

    def step():
        h, mean, rstd = L.layer_norm_forward(x, p["nw"], p["nb"])
        loss, lse = L.linear_cross_entropy_forward(h, p["v"], p["target"], bias=p["vb"])
        dh, dv, db = L.linear_cross_entropy_vjp(h, p["v"], p["target"], lse, torch.ones_like(loss), bias=p["vb"],
                                                want=(True, True, True))
        grads = L.layer_norm_vjp(x, p["nw"], mean, rstd, dh)
        with torch.no_grad():
            return [loss, dv, db, *grads, model(x, p, plan_of, (q1, q2))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x1, p1, _ = model_inputs(T, dtype, seed=10 + i)
        x.copy_(x1)
        p["target"].copy_(p1["target"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), i


def training_step(x, p, plan):
    """The gradients of fresh leaves through autograd, the experts' included."""
    leaves = {k: t.detach().requires_grad_(True) for k, t in dict(p, x=x).items() if t.is_floating_point()}
    rows = leaves["x"]
    loss = model(rows, dict(p, **leaves), lambda h: plan)
    return [loss.detach(), *torch.autograd.grad(loss, list(leaves.values()))]


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_replays_of_a_captured_backward_pass_follow_new_inputs(T, dtype):
    """autograd's own pass through all of them, captured with the leaves made
    inside the capture; every replay against the eager step."""
    x, p, plan_of = model_inputs(T, dtype)
    plan = plan_of(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            training_step(x, p, plan)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = training_step(x, p, plan)
    for i in range(4):
        x1, p1, _ = model_inputs(T, dtype, seed=10 + i)
        for k in p:
            p[k].copy_(p1[k])
        x.copy_(x1)
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(out, training_step(x, p, plan))):
            assert torch.equal(a, b), (i, j)


def test_two_streams_at_once():
    """Steps of two sizes, enqueued in turn on two streams, as each alone."""
    cases = []
    for T, dtype in ((60, torch.bfloat16), (500, torch.float32)):
        x, p, plan_of = model_inputs(T, dtype)
        cases.append((x, p, plan_of(x)))
    want = [training_step(*c) for c in cases]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(6):
        for c, side in zip(cases, sides):
            with torch.cuda.stream(side):
                got.append(training_step(*c))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2])), i


def test_rows_that_are_the_vocabulary_too():
    """One leaf in both places: its gradient is the sum of both."""
    t = torch.randn(70, 40, generator=gen(6))
    target = torch.arange(70).roll(3)
    leaf = t.cuda().requires_grad_(True)
    L.linear_cross_entropy(leaf, leaf, target.cuda(), reduction="sum").backward()
    ref = R.loss(t, t, None, target, "sum", torch.ones(()))
    (dx, dxe), (dw, dwe) = ref["dx"], ref["dw"]
    X.check(leaf.grad, dx + dw, X.rounded(dx + dw, t.dtype, dxe + dwe), "gradient")


def test_broadcast_inputs():
    """A row that stands for many, and the scalar gradient of a sum: as the same
    tensors laid out."""
    row = torch.randn(1, 64, generator=gen(7)).cuda().requires_grad_(True)
    one = torch.full((1,), 1.5, device="cuda", requires_grad=True)
    v = torch.randn(30, 64, generator=gen(8)).cuda()
    target = torch.arange(9, device="cuda")
    L.linear_cross_entropy(L.layer_norm(row.expand(9, 64), one.expand(64)), v, target, reduction="none").sum().backward()
    x, w = row.detach().repeat(9, 1).requires_grad_(True), one.detach().repeat(64).requires_grad_(True)
    L.linear_cross_entropy(L.layer_norm(x, w), v, target, reduction="none").backward(torch.ones(9, device="cuda"))
    assert torch.equal(row.grad, x.grad.sum(0, keepdim=True)) and torch.equal(one.grad, w.grad.sum(0, keepdim=True))


# ---- offsets beyond 32 bits ---------------------------------------------------------

@pytest.mark.slow
def test_norm_and_8_bits_past_2_to_the_31_elements():
    T, D = 270_000, 8192  # 2.2e9 elements
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    for r in range(0, T, 30_000):
        x[r:r + 30_000].normal_()
    w = torch.rand(D, device="cuda") + 0.5
    y, mean, rstd = L.layer_norm_forward(x, w)
    at = torch.tensor([0, 1, T // 2, T - 70_000, T - 2, T - 1], device="cuda")
    few, _, _ = L.layer_norm_forward(x[at], w)
    assert torch.equal(y[at], few)
    dx, _, _ = L.layer_norm_vjp(x, w, mean, rstd, y, want=(True, False, False))
    want, _, _ = L.layer_norm_vjp(x[at], w, mean[at], rstd[at], y[at], want=(True, False, False))
    assert torch.equal(dx[at], want)
    del dx, y
    rows, part = L.expert_quantize(x), L.expert_quantize(x[at])
    assert torch.equal(rows.values.view(torch.uint8)[at], part.values.view(torch.uint8))
    assert torch.equal(L.expert_dequantize(rows)[at], L.expert_dequantize(part))
    # as rows of a product, and as its weights
    plan = L.expert_sort(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    qw = L.expert_quantize(torch.randn(1, 16, D, device="cuda"))
    ys = L.expert_linear_fp8(rows, qw, plan)
    one = L.expert_sort(torch.zeros(6, 1, dtype=torch.int32, device="cuda"), 1)
    assert torch.equal(ys[at], L.expert_linear_fp8(part, qw, one))
    wide = L.ScaledRows(rows.values.reshape(2, T // 2, D), rows.scales.reshape(2, T // 2, D // 128), D)
    two = L.expert_sort(torch.tensor([[0], [1], [1]], dtype=torch.int32, device="cuda"), 2)
    q3 = L.expert_quantize(torch.randn(3, D, device="cuda"))
    ys = L.expert_linear_fp8(q3, wide, two)
    v = L.ScaledRows(part.values[3:].reshape(1, 3, D), part.scales[3:].reshape(1, 3, D // 128), D)
    three = L.expert_sort(torch.zeros(3, 1, dtype=torch.int32, device="cuda"), 1)
    assert torch.equal(ys[1:, at[3:] - T // 2], L.expert_linear_fp8(q3, v, three)[1:])


@pytest.mark.slow
def test_norm_of_a_row_of_more_columns_than_a_launch_has_threads_for():
    """Sums of 2^28 columns' gradients leave in turns of the grid: of one row, dbias
    is dy, and dweight dy times the normalised row."""
    D = 2 ** 28 + 3
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.empty(1, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    _, mean, rstd = L.layer_norm_forward(x)
    _, dw, db = L.layer_norm_vjp(x, None, mean, rstd, dy, want=(False, True, True))
    assert torch.equal(db, dy[0])
    assert torch.equal(dw, (dy.float() * ((x.float() - mean) * rstd)).bfloat16()[0])
    torch.cuda.empty_cache()


@pytest.mark.slow
@pytest.mark.parametrize("T", [8, 200])
def test_loss_of_a_vocabulary_past_2_to_the_31_elements(T):
    """The far end of the weights against the same rows taken alone: entries
    without a share of the sums are masked."""
    V, D = 270_000, 8192
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for r in range(0, V, 30_000):
        w[r:r + 30_000].normal_().mul_(D ** -0.5)
    x = torch.randn(T, D, device="cuda").bfloat16()
    n = 1000
    bias = torch.full((V,), -math.inf, dtype=torch.bfloat16, device="cuda")
    bias[-n:] = 0
    target = torch.randint(V - n, V, (T,), device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, target, bias=bias, reduction="none")
    few, few_lse = L.linear_cross_entropy_forward(x, w[-n:], target - (V - n), reduction="none")
    ref = R.loss(x, w[-n:], None, target - (V - n), "none", torch.ones(T, device="cuda"))
    X.check(loss, *ref["loss"], "loss")
    dx, dw, _ = L.linear_cross_entropy_vjp(x, w, target, lse, torch.ones(T, device="cuda"), bias=bias, reduction="none")
    X.check(dx, *ref["dx"], "dx")
    X.check(dw[-n:], *ref["dw"], "dw")
    assert dw[:-n:1001].abs().max() == 0 and dw[V - n - 1].abs().max() == 0
