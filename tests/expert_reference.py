"""The expert operators by their definitions, in float64 on the CPU, with the
error that the kernels' arithmetic can leave at most, element by element.

u is the unit roundoff of the rows' type (a result is rounded to it once),
EPS that of fp32, in which sums are held: a sum of n terms is off by at most
n EPS times the sum of their magnitudes."""
import math

import torch

EPS = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# a 16-bit result below the type's normal range has only this absolute accuracy
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def topk(p, m, floor=-math.inf, normalize=False):
    """ids (list of lists) and weights (float64)."""
    T, E = p.shape
    ids = torch.full((T, m), -1, dtype=torch.int32)
    w = torch.zeros(T, m, dtype=torch.float64)
    rows = p.double()
    for t in range(T):
        row = rows[t].tolist()
        can = [e for e in range(E) if row[e] > floor]
        can.sort(key=lambda e: (-row[e], e))
        for j, e in enumerate(can[:m]):
            ids[t, j] = e
            w[t, j] = row[e]
    sums = w.sum(1, keepdim=True)
    if normalize:
        w = torch.where(sums > 0, w / sums, torch.zeros_like(w))
    return ids, w, sums[:, 0]


def topk_vjp(ids, w, sums, dw, E, normalize):
    T, m = ids.shape
    dp = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        dot = sum(float(dw[t, i]) * float(w[t, i]) for i in range(m) if ids[t, i] >= 0)
        for j in range(m):
            e = int(ids[t, j])
            if e < 0:
                continue
            g = float(dw[t, j])
            if normalize:
                g = (g - dot) / float(sums[t]) if float(sums[t]) > 0 else 0.0
            dp[t, e] = g
    return dp


def sort(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    used = int(offsets[-1])
    place = torch.full((flat.numel(),), -1, dtype=torch.int64)
    place[order[:used]] = torch.arange(used)
    order = order.clone()
    order[used:] = -1
    return offsets.int(), order.int(), place.reshape(ids.shape).int()


def dispatch(x, order, m):
    xs = torch.zeros(order.numel(), x.shape[1], dtype=x.dtype)
    on = order >= 0
    xs[on] = x[(order[on] // m).long()]
    return xs


def gather(rows, place):
    """rows[place[t, j]] as float64, zeros for empty slots."""
    got = rows.double()[place.clamp(min=0).long()] if rows.shape[0] else torch.zeros(*place.shape, rows.shape[1]).double()
    return torch.where((place >= 0)[:, :, None], got, torch.zeros((), dtype=torch.float64))


def rounded(ref, dtype, err):
    """The tolerance of ref, off by err, once rounded to dtype."""
    return err + U[dtype] * (ref.abs() + err) + TINY[dtype]


def act(z, a):
    if a == "relu":
        return z.clamp(min=0)
    if a == "silu":
        return z * torch.sigmoid(z)
    if a == "gelu":
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2)))
    return z


def slope(z, a):
    if a == "relu":
        return (z > 0).double()
    if a == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if a == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def linear(xs, weight, bias, offsets, a, dys=None):
    """{name: (reference, tolerance)} of ys and, with dys, dxs, dw, db.

    z is a sum of K products and a bias in fp32.  |act'| <= 1.13 and act's
    own evaluation is off by a few EPS of |z| (16 taken).  In the backward
    pass z is kept in fp16 (16-bit rows): off by 2^-11 |z| + 2^-24, and the
    slope, with |act''| <= 1, by as much, plus 32 EPS (1 + |z|) of its own."""
    dt = xs.dtype
    P, K = xs.shape
    E, F, _ = weight.shape
    o = offsets.tolist()
    x, wt = xs.double(), weight.double()
    (ys, ye), (dx, dxe), (dw, dwe), (db, dbe) = [[x.new_zeros(s) for _ in range(2)] for s in
                                                 ((P, F), (P, K), (E, F, K), (E, F))]
    for e in range(E):
        r = slice(o[e], o[e + 1])
        n = o[e + 1] - o[e]
        if n == 0:
            continue
        z = x[r] @ wt[e].t()
        mag = x[r].abs() @ wt[e].abs().t()
        if bias is not None:
            z = z + bias[e].double()
            mag = mag + bias[e].double().abs()
        ze = (K + 2) * EPS * mag
        ys[r] = act(z, a)
        ye[r] = 1.13 * ze + (0 if a == "none" else 16 * EPS * z.abs())
        if dys is None:
            continue
        d = dys[r].double()
        s = slope(z, a)
        if a in ("none", "relu"):  # relu: the tests' z keep away from 0
            se = torch.zeros_like(z)
        else:
            se = ze + 32 * EPS * (1 + z.abs())
            if dt != torch.float32:
                se = se + 2.0 ** -11 * z.abs() + 2.0 ** -24
        dz = d * s
        dze = d.abs() * se
        db[e] = dz.sum(0)
        dbe[e] = dze.sum(0) + (n + 2) * EPS * dz.abs().sum(0)
        if a != "none":  # dz rounded to the rows' type for the products
            dze = dze + U[dt] * (dz.abs() + dze) + TINY[dt]
        dx[r] = dz @ wt[e]
        dxe[r] = dze @ wt[e].abs() + (F + 2) * EPS * (dz.abs() @ wt[e].abs())
        dw[e] = dz.t() @ x[r]
        dwe[e] = dze.t() @ x[r].abs() + (n + 2) * EPS * (dz.abs().t() @ x[r].abs())
    out = {"ys": (ys, rounded(ys, dt, ye))}
    if dys is not None:
        out |= {"dxs": (dx, rounded(dx, dt, dxe)), "dw": (dw, rounded(dw, dt, dwe)), "db": (db, rounded(db, dt, dbe))}
    return out


def check(got, ref, tol, label):
    got, ref, tol = got.detach().cpu().double(), ref.cpu(), tol.cpu()
    assert got.shape == ref.shape, f"{label}: shape {tuple(got.shape)}"
    if got.numel() == 0:
        return
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got.reshape(-1)[i].item()!r}, reference {ref.reshape(-1)[i].item()!r}, "
                             f"tolerance {tol.reshape(-1)[i].item():.3g}")
