"""Measured cases of the expert operators: the step from exact-budget gates to
routed tokens, their experts' products and back.

Five operators, each with its plain form in 32 bits (own = False) and as a
call of this package (own = True):

  topk      the m largest gates of every row: expert ids and weights
  sort      (token, slot) pairs in expert order: offsets, order, places
  dispatch  token rows copied to their pairs' places, and its gradient
  linear    every expert's product with bias and activation, and its gradients
  combine   pairs' rows weighted and summed back per token, and its gradients

A case's "dir" is "fwd" (a serving call) or "step" (forward and backward, as
in training).  The pairs' ids leave a share "drop" of the slots empty (-1),
and with "idle" > 0 that many experts get no token at all.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of a few requests: latency of the smallest calls
        {"name": "topk_decode", "op": "topk", "dir": "fwd", "T": 8, "E": 64, "m": 4, "norm": True},
        # gates of a training batch over an odd number of experts
        {"name": "topk_train", "op": "topk", "dir": "step", "T": 65536, "E": 257, "m": 8, "norm": True},
        # the same two uses of the sort; training drops slots below a gate floor
        {"name": "sort_decode", "op": "sort", "dir": "fwd", "T": 8, "E": 64, "m": 4, "drop": 0.0, "idle": 0},
        {"name": "sort_train", "op": "sort", "dir": "fwd", "T": 65536, "E": 257, "m": 8, "drop": 0.1, "idle": 3},
        # a training batch's rows to their experts and the gradient back
        {"name": "dispatch_train", "op": "dispatch", "dir": "step", "T": 16384, "D": 2048, "E": 8, "m": 2, "drop": 0.0,
         "idle": 0, "type": "bf16"},
        # a small odd batch with rows that are no multiple of 16 bytes
        {"name": "dispatch_odd", "op": "dispatch", "dir": "step", "T": 1000, "D": 1001, "E": 5, "m": 3, "drop": 0.3,
         "idle": 1, "type": "f32"},
        # a decode step's rows back to their tokens, residual added
        {"name": "combine_decode", "op": "combine", "dir": "fwd", "T": 4, "D": 4096, "E": 64, "m": 8, "drop": 0.0,
         "idle": 0, "type": "bf16", "residual": True},
        # a training batch back to its tokens, gradients of rows and weights
        {"name": "combine_train", "op": "combine", "dir": "step", "T": 16384, "D": 2048, "E": 64, "m": 4, "drop": 0.05,
         "idle": 0, "type": "bf16", "residual": True},
        # a decode step's products: every chosen expert's weights are read for a few rows
        {"name": "linear_decode", "op": "linear", "dir": "fwd", "T": 16, "K": 2048, "F": 1024, "E": 64, "m": 4,
         "drop": 0.0, "idle": 0, "type": "bf16", "bias": True, "act": "silu"},
        # a prompt's products with many rows for each expert
        {"name": "linear_prefill", "op": "linear", "dir": "fwd", "T": 8192, "K": 1024, "F": 4096, "E": 16, "m": 2,
         "drop": 0.0, "idle": 0, "type": "f16", "bias": True, "act": "gelu"},
        # a training step of the experts' first layer: the largest case
        {"name": "linear_train", "op": "linear", "dir": "step", "T": 16384, "K": 2048, "F": 4096, "E": 8, "m": 2,
         "drop": 0.02, "idle": 0, "type": "bf16", "bias": True, "act": "silu"},
        # small odd layers in 32 bits, an expert without tokens
        {"name": "linear_odd", "op": "linear", "dir": "step", "T": 513, "K": 257, "F": 1001, "E": 7, "m": 2, "drop": 0.2,
         "idle": 1, "type": "f32", "bias": True, "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges: sizes spread over their
    logarithm, odd ones among them, every type and direction."""
    op = rng.choice(["topk", "sort", "dispatch", "linear", "linear", "combine"])
    E = _log(rng, 4, 257)
    m = rng.randint(1, min(8, E - 1))
    c = {"op": op, "dir": rng.choice(["fwd", "step"]), "E": E, "m": m}
    if op == "topk":
        return c | {"T": _log(rng, 1, 65536), "norm": rng.random() < 0.5}
    c |= {"drop": rng.choice([0.0, 0.05, 0.3]), "idle": rng.choice([0, 0, 1, 2]) if E - m > 2 else 0}
    if op == "sort":
        return c | {"dir": "fwd", "T": _log(rng, 1, 65536)}
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    # widths: multiples of 64, of 8, and any
    unit = rng.choice([64, 64, 8, 1])

    def width(lo, hi):
        return max(1, _log(rng, lo, hi) // unit) * unit

    if op in ("dispatch", "combine"):
        c |= {"D": width(64, 4096), "type": kind}
        c["T"] = _log(rng, 1, max(1, min(65536, (1 << 27) // (c["D"] * m))))
        return c | ({"residual": rng.random() < 0.5} if op == "combine" else {})
    # relu forward only: its slope jumps at 0, where two right sums may fall on either side
    c |= {"K": width(64, 4096), "F": width(64, 4096), "type": kind, "bias": rng.random() < 0.7,
          "act": rng.choice(["none", "silu", "gelu"] + (["relu"] if c["dir"] == "fwd" else []))}
    while E * c["K"] * c["F"] > 1 << 28:  # weights within 512 MiB in 16 bits
        E = max(2, E // 2)
        c |= {"E": E, "m": min(m, E - 1), "idle": 0}
    # 32-bit products run at a sixteenth of the 16-bit rate
    pairs = (1 << 38 if kind != "f32" else 1 << 34) // (c["K"] * c["F"])
    c["T"] = _log(rng, 1, max(1, min(32768, pairs) // c["m"]))
    return c


def _ids(case, gen):
    """Distinct experts of every token: a random choice with uneven loads,
    idle experts never chosen, dropped slots -1."""
    T, E, m = case["T"], case["E"], case["m"]
    load = torch.rand(E, generator=gen, device="cuda") + 0.5
    if case["idle"]:
        load[torch.randperm(E, generator=gen, device="cuda")[:case["idle"]]] = 0.0
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-9, 1 - 1e-7)))
    ids = (load.log() + noise).topk(m, dim=1).indices.to(torch.int32)
    if case["drop"]:
        ids[torch.rand(T, m, generator=gen, device="cuda") < case["drop"]] = -1
    return ids


def _plan(ids, E):
    """offsets, order and places of the pairs, by elementary operations."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=ids.device)[None, :]).sum(0) if flat.numel() * E < 1 << 22 \
        else torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=ids.device)
    place = torch.where(flat < 0, torch.full_like(place, -1), place)
    pos = torch.arange(flat.numel(), device=ids.device)
    order = torch.where(pos < offsets[-1], order, torch.full_like(order, -1))
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32).reshape(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, E, m = case["T"], case["E"], case["m"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale)

    s = {"case": case}
    if case["op"] == "topk":
        # gates as the row solve leaves them: most near 0, a few near 1
        s["p"] = torch.sigmoid(normal(T, E, scale=2.0) - 2.0)
        s["dw"] = normal(T, m)
        return s
    ids = _ids(case, gen)
    s["ids"] = ids
    if case["op"] == "sort":
        return s
    kind = DTYPES[case["type"]]
    s["offsets"], s["order"], s["place"] = _plan(ids, E)
    P = T * m
    if case["op"] == "dispatch":
        s["x"] = normal(T, case["D"]).to(kind)
        s["dxs"] = normal(P, case["D"]).to(kind)
    elif case["op"] == "combine":
        s["ys"] = normal(P, case["D"]).to(kind)
        s["w"] = torch.rand(T, m, generator=gen, device="cuda")
        s["residual"] = normal(T, case["D"]).to(kind) if case["residual"] else None
        s["dout"] = normal(T, case["D"]).to(kind)
    else:
        K, F = case["K"], case["F"]
        s["xs"] = normal(P, K).to(kind)
        s["xs"][int(s["offsets"][-1]):] = 0  # as dispatch leaves the unused places
        s["weight"] = torch.empty(E, F, K, dtype=kind, device="cuda")
        for e in range(E):
            s["weight"][e] = normal(F, K, scale=K ** -0.5).to(kind)
        s["bias"] = normal(E, F, scale=0.5).to(kind) if case["bias"] else None
        s["dys"] = normal(P, F).to(kind)
        # the row capacity the plain form pads every expert to
        s["cap"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    return s


# ---- plain forms -------------------------------------------------------------

def _plain_topk(s):
    p, case = s["p"], s["case"]
    # the m largest, ties to the lowest index: a stable descending sort
    w, ids = torch.sort(p, dim=1, descending=True, stable=True)
    w, ids = w[:, :case["m"]], ids[:, :case["m"]]
    total = w.sum(1, keepdim=True)
    out = w / total if case["norm"] else w
    if case["dir"] == "fwd":
        return ids.to(torch.int32), out.contiguous()
    g = s["dw"]
    if case["norm"]:
        g = (g - (g * out).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(p).scatter(1, ids, g)
    return ids.to(torch.int32), out.contiguous(), dp


def _plain_dispatch(s):
    case = s["case"]
    used = s["order"] >= 0
    token = torch.where(used, s["order"] // case["m"], 0).long()
    xs = torch.where(used[:, None], s["x"][token], torch.zeros((), dtype=s["x"].dtype, device="cuda"))
    if case["dir"] == "fwd":
        return xs
    place = s["place"].long()
    rows = s["dxs"][place.clamp(min=0)].float() * (place >= 0)[:, :, None]
    return xs, rows.sum(1).to(s["x"].dtype)


def _plain_combine(s):
    case = s["case"]
    place = s["place"].long()
    on = place >= 0
    w = s["w"] * on
    rows = s["ys"][place.clamp(min=0)].float()
    out = (rows * w[:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    out = out.to(s["ys"].dtype)
    if case["dir"] == "fwd":
        return out
    dout = s["dout"].float()
    dw = (rows * dout[:, None, :]).sum(2) * on
    used = s["order"] >= 0
    pair = s["order"].clamp(min=0).long()
    dys = dout[pair // case["m"]] * (w.reshape(-1)[pair] * used)[:, None]
    return out, dys.to(s["ys"].dtype), dw


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _plain_linear(s):
    """One batched product over the experts, their rows padded to one length."""
    case = s["case"]
    xs, weight, off = s["xs"], s["weight"].float(), s["offsets"].long()
    slot = torch.arange(max(1, s["cap"]), device="cuda")
    row = off[:-1, None] + slot[None, :]                    # [E, cap]
    on = row < off[1:, None]
    row = row.clamp(max=xs.shape[0] - 1)
    x = xs[row].float() * on[:, :, None]
    z = torch.bmm(x, weight.transpose(1, 2).contiguous())
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None, :]
    y = torch.zeros(xs.shape[0], case["F"], dtype=xs.dtype, device="cuda")
    y[row[on]] = _act(z, case["act"]).to(xs.dtype)[on]
    if case["dir"] == "fwd":
        return y
    dz = s["dys"][row].float() * on[:, :, None] * _act_grad(z, case["act"])
    dx = torch.zeros_like(xs)
    dx[row[on]] = torch.bmm(dz, weight).to(xs.dtype)[on]
    dw = torch.bmm(dz.transpose(1, 2).contiguous(), x).to(xs.dtype)
    out = (y, dx, dw)
    return out + (dz.sum(1).to(xs.dtype),) if s["bias"] is not None else out


def _plain(s):
    op, case = s["case"]["op"], s["case"]
    if op == "topk":
        return _plain_topk(s)
    if op == "sort":
        return _plan(s["ids"], case["E"])
    if op == "dispatch":
        return _plain_dispatch(s)
    if op == "combine":
        return _plain_combine(s)
    return _plain_linear(s)


# ---- the package's operators ---------------------------------------------------

def _own(s):
    import differentiable_exact_budget_amd as L

    case = s["case"]
    op, step = case["op"], case["dir"] == "step"
    if op == "topk":
        p = s["p"].detach().requires_grad_(step)
        ids, w = L.expert_topk(p, case["m"], normalize=case["norm"])
        return (ids, w.detach(), torch.autograd.grad(w, p, s["dw"])[0]) if step else (ids, w)
    if op == "sort":
        plan = L.expert_sort(s["ids"], case["E"])
        return plan.offsets, plan.order, plan.place
    plan = L.ExpertPlan(case["E"], s["offsets"], s["order"], s["place"])
    if op == "dispatch":
        x = s["x"].detach().requires_grad_(step)
        xs = L.expert_dispatch(x, plan)
        return (xs.detach(), torch.autograd.grad(xs, x, s["dxs"])[0]) if step else xs
    if op == "combine":
        ys, w = s["ys"].detach().requires_grad_(step), s["w"].detach().requires_grad_(step)
        out = L.expert_combine(ys, w, plan, residual=s["residual"])
        return (out.detach(), *torch.autograd.grad(out, (ys, w), s["dout"])) if step else out
    leaves = [t.detach().requires_grad_(step) for t in (s["xs"], s["weight"], s["bias"]) if t is not None]
    y = L.expert_linear(leaves[0], leaves[1], plan, bias=leaves[2] if len(leaves) > 2 else None,
                        activation=case["act"])
    return (y.detach(), *torch.autograd.grad(y, leaves, s["dys"])) if step else y


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    op, T, E, m, step = case["op"], case["T"], case["E"], case["m"], case["dir"] == "step"
    P = T * m
    if op == "topk":
        b = 4 * T * E + 8 * P
        return {"bytes": b + (4 * P + 4 * T * E if step else 0), "flops": T * E}
    if op == "sort":
        return {"bytes": 12 * P + 4 * (E + 1), "flops": P}
    size = 4 if case["type"] == "f32" else 2
    live = P * (1 - case["drop"])
    if op == "dispatch":
        D = case["D"]
        b = (T + P) * D * size + 4 * P
        return {"bytes": b + ((live + T) * D * size + 4 * P if step else 0), "flops": live * D if step else 0}
    if op == "combine":
        D = case["D"]
        b = (live + T + (T if case["residual"] else 0)) * D * size + 8 * P
        back = (T + P + live) * D * size + 12 * P
        return {"bytes": b + (back if step else 0), "flops": (2 + (3 if step else 0)) * live * D}
    K, F = case["K"], case["F"]
    busy = max(1, E - case["idle"])
    active = busy * (1 - (1 - min(1.0, m * (1 - case["drop"]) / busy)) ** T)
    b = active * F * (K + (1 if case["bias"] else 0)) * size + live * K * size + P * F * size
    back = live * (F + K) * size + active * F * K * size + P * K * size + E * F * K * size
    return {"bytes": b + (back if step else 0), "flops": (6 if step else 2) * live * K * F}


# ---- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, step, m, E = case["op"], case["dir"] == "step", case["m"], case["E"]
    if op == "sort":
        return None
    if op == "topk":
        p = s["p"].double()
        T = p.shape[0]
        left, chosen = p.clone(), []
        lanes = torch.arange(E, device="cuda").expand(T, E)
        for _ in range(m):
            top = left.max(1, keepdim=True).values
            first = torch.where(left == top, lanes, E).min(1, keepdim=True).values
            chosen.append(first)
            left.scatter_(1, first, -math.inf)
        ids = torch.cat(chosen, 1)
        v = p.gather(1, ids)
        total = v.sum(1, keepdim=True)
        w = v / total if case["norm"] else v
        if not step:
            return None, w
        # d w_i / d v_j = (delta_ij - w_i) / total with normalised weights
        jac = torch.eye(m, dtype=torch.float64, device="cuda").expand(T, m, m)
        if case["norm"]:
            jac = (jac - w[:, :, None]) / total[:, :, None]
        dv = (s["dw"].double()[:, :, None] * jac).sum(1)
        dp = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        dp.scatter_add_(1, ids, dv)
        return None, w, dp
    off = s["offsets"].tolist()
    total = off[-1]
    if op == "dispatch":
        D, T = case["D"], case["T"]
        token = (s["order"][:total] // m).long()
        xs = torch.zeros(T * m, D, dtype=torch.float64, device="cuda")
        xs[:total] = s["x"].double()[token]
        if not step:
            return xs
        dx = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        for j in range(m):
            at = s["place"][:, j].long()
            hit = (at >= 0).nonzero()[:, 0]
            dx[hit] += s["dxs"][at[hit]].double()
        return xs, dx
    if op == "combine":
        D, T = case["D"], case["T"]
        out = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            out += s["residual"].double()
        dys = torch.zeros(T * m, D, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, m, dtype=torch.float64, device="cuda")
        for j in range(m):
            at = s["place"][:, j].long()
            hit = (at >= 0).nonzero()[:, 0]
            at = at[hit]
            y, w, g = s["ys"][at].double(), s["w"][hit, j].double()[:, None], s["dout"][hit].double()
            out[hit] += w * y
            dys[at] = w * g
            dw[hit, j] = (y * g).sum(1)
        return (out, dys, dw) if step else out
    K, F, P = case["K"], case["F"], case["T"] * m
    y = torch.zeros(P, F, dtype=torch.float64, device="cuda")
    dx = torch.zeros(P, K, dtype=torch.float64, device="cuda") if step else None
    dw = torch.zeros(E, F, K, dtype=torch.float64, device="cuda") if step else None
    db = torch.zeros(E, F, dtype=torch.float64, device="cuda") if step else None
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x, weight = s["xs"][a:b].double(), s["weight"][e].double()
        z = x @ weight.t()
        if s["bias"] is not None:
            z = z + s["bias"][e].double()
        q = 0.5 * (1 + torch.erf(z / math.sqrt(2.0)))
        g = 1 / (1 + torch.exp(-z))
        y[a:b] = {"none": z, "relu": torch.relu(z), "silu": z * g, "gelu": z * q}[case["act"]]
        if not step:
            continue
        slope = {"none": torch.ones_like(z), "relu": (z > 0).double(), "silu": g + z * g * (1 - g),
                 "gelu": q + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)}[case["act"]]
        dz = s["dys"][a:b].double() * slope
        dx[a:b] = dz @ weight
        dw[e] = dz.t() @ x
        db[e] = dz.sum(0)
    if not step:
        return y
    return (y, dx, dw, db) if s["bias"] is not None else (y, dx, dw)
