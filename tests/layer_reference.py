"""The norm, the loss and the experts' products in 8 bits by their definitions,
in float64, with the error that the kernels' arithmetic can leave at most,
element by element (u and EPS as in expert_reference)."""
import math

import torch

from expert_reference import EPS, TINY, U, act, rounded

BLOCK = 128


def norm(x, weight, bias, eps, dy=None):
    """{name: (reference, tolerance)} of y, mean, rstd and, with dy, dx, dw, db.

    A row's sums run over at most 32 elements a thread (or its share of a row
    that registers do not hold), then over lanes and waves: a depth of 64 and a
    share more.  A mean that is off by m shifts all of a row's differences alike:
    their squares are off by m^2 each, since the differences themselves sum to 0,
    and by their own roundings."""
    dt = x.dtype
    T, D = x.shape
    wt = dt if weight is None else weight.dtype
    depth = 64 + D / 1024
    xd = x.double()
    w = torch.ones(D, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(D, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    mean = xd.mean(1, keepdim=True)
    me = depth * EPS * xd.abs().mean(1, keepdim=True)
    diff = xd - mean
    var = diff.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    # differences rounded once each, squares and their sum
    ve = (depth + 8) * EPS * var + me.square() * 2 + 4 * EPS * me * diff.abs().mean(1, keepdim=True)
    rel = 0.5 * ve * rstd.square() + 6 * EPS
    xh = diff * rstd
    xe = xh.abs() * (rel + 4 * EPS) + me * rstd
    y = xh * w + b
    out = {"y": (y, rounded(y, dt, xe * w.abs() + 2 * EPS * ((xh * w).abs() + y.abs()))),
           "mean": (mean[:, 0], (me + EPS * mean.abs())[:, 0]), "rstd": (rstd[:, 0], (rstd * rel)[:, 0])}
    if dy is None:
        return out
    d = dy.double()
    g = d * w
    s1, s2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    s1e = (depth + 4) * EPS * g.abs().mean(1, keepdim=True)
    s2e = (g.abs() * xe).mean(1, keepdim=True) + (depth + 6) * EPS * (g * xh).abs().mean(1, keepdim=True)
    dx = rstd * (g - s1 - xh * s2)
    dxe = rstd * (s1e + xh.abs() * s2e + xe * s2.abs() + 8 * EPS * (g.abs() + s1.abs() + (xh * s2).abs())) + rel * dx.abs()
    dw, db = (d * xh).sum(0), d.sum(0)
    dwe = (d.abs() * xe).sum(0) + (T + 8) * EPS * (d * xh).abs().sum(0)
    dbe = (T + 8) * EPS * d.abs().sum(0)
    return out | {"dx": (dx, rounded(dx, dt, dxe)), "dw": (dw, rounded(dw, wt, dwe)), "db": (db, rounded(db, wt, dbe))}


def loss(x, weight, bias, target, reduction, dloss=None):
    """{name: (reference, tolerance)} of loss, lse and, with dloss, dx, dw, db.

    z is a sum of D products and a bias in fp32.  The sum of exponentials is
    taken in parts, at most 64 + V / 16 deep; an exponential is off by 2 ulp and by
    its argument's rounding, 3 EPS a of a term e^-a, which is at most 1.2 EPS of the
    sum.  d, over the largest gradient of a row, is rounded to 16-bit types
    once (in fp16 times 2^13, so that 2^-38 of that gradient is the least)."""
    dt = x.dtype
    D, V = x.shape[1], weight.shape[0]
    T = x.shape[0]
    xd, w = x.double(), weight.double()
    z = xd @ w.t()
    mag = xd.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + torch.where(bias.isfinite(), bias.double(), 0.0).abs()
    ze = (D + 2) * EPS * mag
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    # an error of z moves the logarithm by its mean under p
    le = (p * ze).sum(1) + (80 + V / 16) * EPS + 4 * EPS * lse.abs()
    on = (target >= 0) & (target < V)
    at = target.clamp(0, V - 1)[:, None]
    zt = z.gather(1, at)[:, 0]
    each = torch.where(on, lse - zt, 0.0)
    ee = torch.where(on, le + ze.gather(1, at)[:, 0] + 2 * EPS * each.abs(), 0.0)
    count = max(1, int(on.sum())) if reduction == "mean" else 1
    out = {"lse": (lse, le + 2 * EPS * lse.abs())}
    if reduction == "none":
        out["loss"] = (each, ee)
    else:
        out["loss"] = (each.sum() / count, ee.sum() / count + 2 * EPS * each.sum().abs() / count)
    if dloss is None:
        return out
    g = torch.where(on, dloss.double() / count, 0.0)
    hot = torch.zeros_like(z).scatter_(1, at, 1.0)
    d = (p - hot) * g[:, None]
    gap = torch.where(z.isfinite(), z - lse[:, None], 0.0).abs()
    de = (p * (ze + le[:, None] + (4 + 3 * gap) * EPS) + 4 * EPS * (p - hot).abs()) * g.abs()[:, None]
    if dt != torch.float32:
        de = de + U[dt] * (d.abs() + de) + (2.0 ** -37 * g.abs().max() if dt == torch.float16 and T else 0)
        de = de * (g != 0)[:, None]
    dx, dw, db = d @ w, d.t() @ xd, d.sum(0)
    dxe = de @ w.abs() + (V + 8) * EPS * (d.abs() @ w.abs())
    dwe = de.t() @ xd.abs() + (T + 8) * EPS * (d.abs().t() @ xd.abs())
    dbe = de.sum(0) + (T + 8) * EPS * d.abs().sum(0)
    return out | {"dx": (dx, rounded(dx, dt, dxe)), "dw": (dw, rounded(dw, dt, dwe)), "db": (db, rounded(db, dt, dbe))}


# the magnitudes that e4m3 holds
E4M3 = sorted({m * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in
               ([8 + i for i in range(8)] if e else range(8)) if not (e == 15 and m == 15)})


def quantize(x):
    """(values, exponents) of rows in 8 bits, float64 and int: by search in the
    list of what e4m3 holds."""
    *lead, D = x.shape
    blocks = -(-D // BLOCK)
    rows = torch.zeros(math.prod(lead), blocks * BLOCK, dtype=torch.float64)
    rows[:, :D] = x.double().reshape(-1, D)
    rows = rows.reshape(-1, BLOCK)
    finite = rows.isfinite()
    top = torch.where(finite, rows, 0.0).abs().amax(1)
    e = torch.zeros(rows.shape[0], dtype=torch.int64)
    for i, t in enumerate(top.tolist()):
        if t > 0:
            k = math.frexp(t)[1] - 10
            while t > math.ldexp(448.0, k):
                k += 1
            e[i] = max(k, -127)
    u = rows * torch.exp2(-e.double())[:, None]
    table = torch.tensor(E4M3, dtype=torch.float64)
    mag = torch.where(finite, u, 0.0).abs()
    hi = torch.searchsorted(table, mag).clamp(max=len(E4M3) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = mag - table[lo], table[hi] - mag
    # ties to the even mantissa, which is the even place in the list
    take = torch.where(below < above, lo, torch.where(above < below, hi, torch.where(lo % 2 == 0, lo, hi)))
    take = torch.where(table[hi] == mag, hi, take)
    q = torch.copysign(table[take], u)
    q = torch.where(finite, q, math.nan)
    return q.reshape(*lead, blocks * BLOCK), e.reshape(*lead, blocks)


def stands_for(values, exponents, width):
    """What rows in 8 bits stand for (float64)."""
    v = values.unflatten(-1, (-1, BLOCK)) * torch.exp2(exponents.double())[..., None]
    return v.flatten(-2)[..., :width]


def linear8(xs, weight, bias, offsets, a, dtype):
    """(reference, tolerance) of ys from what the rows and weights stand for.

    For 16-bit results the matrix instruction drops from each product of eight
    neighbours what is below 2^-13 of the largest one's power of two: seven times
    that is lost at most.  For float32 results the operands are in bf16, which
    holds e4m3's four bits down to its least step, 2^-133, of which a smaller
    number keeps the nearest multiple: each operand is off by 2^-134 at most, which
    counts by the other one's magnitude."""
    groups = lambda v: torch.nn.functional.pad(v.abs(), (0, -v.shape[-1] % 8)).unflatten(-1, (-1, 8)).amax(-1)  # noqa: E731
    P, K = xs.shape
    E, F, _ = weight.shape
    o = offsets.tolist()
    y = xs.new_zeros(P, F)
    err = xs.new_zeros(P, F)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        z = xs[r] @ weight[e].t()
        mag = xs[r].abs() @ weight[e].abs().t()
        if bias is not None:
            z = z + bias[e].double()
            mag = mag + bias[e].double().abs()
        y[r] = act(z, a)
        if dtype != torch.float32:
            lost = 7 * 2.0 ** -13 * (groups(xs[r]) @ groups(weight[e]).t()) if K else 0
        else:
            lost = 2.0 ** -134 * (xs[r].abs().sum(1, keepdim=True) + weight[e].abs().sum(1))
        err[r] = 1.13 * ((K + 2) * EPS * mag + lost) + (0 if a == "none" else 16 * EPS * z.abs())
        if a == "gelu" and dtype != torch.float32:  # the polynomial tail, 2.1e-4 Q(|z|) off at most
            err[r] += 2.2e-4 * z.abs() * 0.5 * torch.erfc(z.abs() / math.sqrt(2)) + 4e-7 * z.abs()
    return y, rounded(y, dtype, err)
