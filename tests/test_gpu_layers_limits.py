"""The norm, the loss and the experts' products in 8 bits at their limits: rows
that take no part and hold anything, results of nothing, and sizes that take the
kernels' rarer paths."""
import math

import pytest
import torch

import expert_reference as X
import layer_reference as R
from test_gpu_layers import L, TYPES, check_loss, check_norm, gen, loss_case, norm_case, put

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


# ---- norm rows whose sums pass float32's range ---------------------------------------

# every shape of a row: a wave's, a workgroup's, and what registers do not hold
WIDTHS = [2, 3, 300, 1001, 4096, 5000, 8192, 16384, 20001]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_norm_of_large_values_of_one_sign(dtype, D):
    """Rows whose sum passes float32's range.  Of one value: the variance is 0 and
    that value the mean, so y is the bias.  With a variance past the range: rstd is 0,
    y the bias, and the gradient 0; the mean is as near as any sum of D.  The rows
    between stay as they are."""
    x, w, b, dy = norm_case(9, D, dtype, dtype)
    want, mean0, rstd0 = L.layer_norm_forward(*put(x, w, b))
    dx0, _, _ = L.layer_norm_vjp(*put(x, w), mean0, rstd0, dy.cuda())
    big = torch.finfo(dtype).max
    x[1], x[3] = 3e38, -big
    x[5] = (2e38 * (1 + 0.2 * torch.randn(D, generator=gen(1)).clamp(-3, 3))).to(dtype)
    x[7] = torch.where(torch.arange(D) % 3 == 0, -big, big).to(dtype)
    y, mean, rstd = L.layer_norm_forward(*put(x, w, b))
    dx, dw, db = L.layer_norm_vjp(*put(x, w), mean, rstd, dy.cuda())
    assert dw.isfinite().all() and db.isfinite().all()
    for r in range(9):
        if r % 2 == 0:
            assert torch.equal(y[r], want[r]) and torch.equal(dx[r], dx0[r])
            assert mean[r] == mean0[r] and rstd[r] == rstd0[r]
            continue
        assert torch.equal(y[r].cpu(), b), r
        true = float(x[r].double().mean())
        if r < 4:
            assert float(mean[r]) == true and abs(float(rstd[r]) - 1e-5 ** -0.5) < 1e-3
        else:
            depth = 64 + D / 1024  # of a row's sums
            assert rstd[r] == 0 and not dx[r].any()
            assert abs(float(mean[r]) - true) <= depth * 2.0 ** -24 * float(x[r].double().abs().mean())


@pytest.mark.parametrize("D", [d for d in WIDTHS if d >= 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_norm_of_variances_whose_sums_pass_float32(dtype, D):
    """Values about 1.5e18: D squares are past float32's range, their mean is not."""
    x, w, b, dy = norm_case(5, D, dtype, dtype)
    x[1], x[4] = (1.5e18 * (torch.randn(2, D, generator=gen(2)) + 0.5)).to(dtype)
    assert float(x[1].double().var()) * D > 3.5e38
    check_norm(x, w, b, dy)


# ---- gradients without elements --------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_without_elements_are_empty(dtype):
    """No rows, or no width, where those are the only gradients that are wanted."""
    on = {"device": "cuda", "dtype": dtype}
    x = torch.empty(0, 16, **on, requires_grad=True)
    assert torch.autograd.grad(L.layer_norm(x).sum(), x)[0].shape == (0, 16)
    y, mean, rstd = L.layer_norm_forward(x)
    assert L.layer_norm_vjp(x, None, mean, rstd, y, want=(True, False, False))[0].shape == (0, 16)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    loss = L.linear_cross_entropy(x, torch.rand(30, 16, **on), none)
    assert torch.autograd.grad(loss, x)[0].shape == (0, 16)
    e, w = torch.empty(5, 0, **on, requires_grad=True), torch.empty(30, 0, **on, requires_grad=True)
    target = torch.arange(5, device="cuda")
    dx, dw = torch.autograd.grad(L.linear_cross_entropy(e, w, target), (e, w))
    assert dx.shape == (5, 0) and dw.shape == (30, 0)
    _, lse = L.linear_cross_entropy_forward(e, w, target)
    got = L.linear_cross_entropy_vjp(e, w, target, lse, torch.ones((), device="cuda"))
    assert got[0].shape == (5, 0) and got[1].shape == (30, 0) and got[2] is None


# ---- the bias' gradient -----------------------------------------------------------------

def check_db(x, w, b, target):
    """db, whose sums are of d as it is in float32: what float32 rows may be off by,
    and the result's rounding to its own type."""
    leaves = [t.cuda() for t in (x, w, b)]
    loss, lse = L.linear_cross_entropy_forward(leaves[0], leaves[1], target.cuda(), bias=leaves[2])
    scale = torch.full((), 512.0 if x.dtype == torch.float16 else 1.0)
    got = L.linear_cross_entropy_vjp(leaves[0], leaves[1], target.cuda(), lse, scale.cuda(), bias=leaves[2],
                                     want=(True, True, True))
    alone = L.linear_cross_entropy_vjp(leaves[0], leaves[1], target.cuda(), lse, scale.cuda(), bias=leaves[2],
                                       want=(False, False, True))
    assert torch.equal(alone[2], got[2])
    fine = [t.float() for t in leaves]
    db, tol = R.loss(fine[0], fine[1], fine[2], target.cuda(), "mean", scale.cuda())["db"]
    X.check(got[2], db, X.rounded(db, x.dtype, tol), "db")


@pytest.mark.parametrize("T,D", [(11, 64), (22, 64), (66, 64), (660, 72), (11, 33), (66, 33)])
@pytest.mark.parametrize("dtype", TYPES)
def test_bias_gradients_that_cancel(dtype, T, D):
    """Every entry of eleven has an eleventh of each row's softmax and is the target
    of an eleventh of the rows: the gradient is 0, which sums of 1/11 and -10/11
    rounded to 16 bits are not."""
    x, w, b = torch.zeros(T, D, dtype=dtype), torch.ones(11, D, dtype=dtype), torch.zeros(11, dtype=dtype)
    check_db(x, w, b, torch.arange(T) % 11)


@pytest.mark.parametrize("T,V,D", [(30, 1000, 64), (300, 3001, 136), (3100, 4001, 64), (1100, 2100, 129), (90, 501, 33)])
@pytest.mark.parametrize("dtype", TYPES)
def test_bias_gradients(dtype, T, V, D):
    check_db(*loss_case(T, V, D, dtype))


# ---- the loss' rarer paths ------------------------------------------------------------

CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def up256(n):
    return -(-n // 256) * 256


def tile_scratch(T, V, D):
    """(pieces, scratch bytes) of the gradient's plan for 16-bit rows on 16 bytes."""
    columns = lambda size: size // 2 // T // 256 * 256  # noqa: E731
    fill = -(-(1 << 24) // (256 * D)) * 256
    width = min(max(columns(256 << 20), min(fill, columns(1 << 30)), 256), 1 << 18, V)
    ld, pieces = -(-width // 8) * 8, -(-V // width)
    shares = max(1, min(512 // (-(-T // 64) * -(-D // 64)), width // 512))
    size = up256((T + 1) * 4) + up256(T * D * 2) + up256(T * ld * 2) + up256(max(2 * -(-T // 64), 4) * ld * 4)
    return pieces, size + (up256(shares * T * D * 4) if pieces * shares > 1 else 0)


def any_scratch(T, V, D):
    """The same of odd widths, with one share of a piece."""
    width = min(max((128 << 20) // 4 // T // 128 * 128, 128), V)
    pieces = -(-V // width)
    size = up256((T + 1) * 4) + up256(T * D * 2) + up256(T * width * 2) + up256(-(-T // 32) * 16 * width)
    return pieces, size + (up256(T * D * 4) if pieces > 1 else 0)


def loss_in_chunks(x, w, b, target, dloss, rows):
    """The gradients of a mean and their tolerances, `rows` rows at a time: those of
    dw and db with a rounding for every chunk."""
    count = max(1, int(((target >= 0) & (target < w.shape[0])).sum()))
    dx, dw, db = [], 0, 0
    for r in range(0, x.shape[0], rows):
        ref = R.loss(x[r:r + rows], w, b, target[r:r + rows], "sum", dloss / count)
        dx.append(torch.stack(ref["dx"]))
        dw, db = dw + torch.stack(ref["dw"]), db + torch.stack(ref["db"])
    return torch.cat(dx, 1), dw, db


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("T,V,D,scratch", [(524_003, 2500, 8, tile_scratch), (200_003, 300, 9, any_scratch)])
def test_gradients_in_three_pieces_of_the_vocabulary(dtype, T, V, D, scratch):
    """Every piece with a share of each row's softmax, and the last one ragged."""
    pieces, size = scratch(T, V, D)
    assert pieces == 3
    assert L.layers.lib().lapsum_linear_cross_entropy_vjp_scratch_bytes(CODE[dtype], T, V, D) == size
    x, w, b, target = put(*loss_case(T, V, D, dtype, drop=0.5))
    leaves = [t.requires_grad_(True) for t in (x, w, b)]
    dloss = torch.full((), 1024.0 if dtype == torch.float16 else 1.0, device="cuda")
    loss = L.linear_cross_entropy(x, w, target, bias=b)
    got = torch.autograd.grad(loss, leaves, dloss)
    for name, a, (value, tol) in zip(("dx", "dw", "db"), got, loss_in_chunks(
            x.detach(), w.detach(), b.detach(), target, dloss, 50_000)):
        X.check(a, value, tol, name)


# odd widths on wide tiles; the widest tiles of the forward pass and of d over several
# steps, and with a last round cut into quarters, one of which has no columns; the
# widest of dx (cut, in two pieces) and of dw
@pytest.mark.parametrize("T,V,D", [(1100, 2100, 129), (4096, 3601, 200), (1024, 16465, 72), (16_700, 17_000, 1024)])
@pytest.mark.parametrize("dtype", TYPES[1:])
def test_losses_on_wide_tiles(dtype, T, V, D):
    check_loss(*put(*loss_case(T, V, D, dtype)), on="cuda")


def test_odd_rows_off_16_bytes_on_wide_tiles():
    """Widths of whole 16 bytes at an address that is not."""
    x, w, b, target = loss_case(1100, 2100, 128, torch.bfloat16)
    want = check_loss(x, w, b, target, on="cuda")
    off = [torch.cat([t.new_zeros(1), t.reshape(-1)]).cuda()[1:].reshape(t.shape).requires_grad_(True) for t in (x, w, b)]
    assert off[0].data_ptr() % 16 == 2
    L.linear_cross_entropy(off[0], off[1], target.cuda(), bias=off[2]).backward(torch.rand((), generator=gen(5)).cuda() + 0.5)
    ref = R.loss(*(t.cuda() for t in (x, w, b, target)), "mean", torch.rand((), generator=gen(5)).cuda() + 0.5)
    for name, t, u in zip(("dx", "dw", "db"), off, want):
        X.check(t.grad, *ref[name], name)
        assert t.grad.shape == u.grad.shape
