"""Measured cases of the operators around a routed layer: the norm in front of
it, the loss behind it, and its experts' products in 8 bits.

Four operators, each with its plain form in 32 bits (own = False) and as a
call of this package (own = True):

  norm     layer norm of rows, and its gradients
  loss     softmax cross entropy of a product with a vocabulary's weights,
           and its gradients
  quant    rows to 8-bit floating point with a power-of-two scale for each
           block of 128, and read back
  linear8  every expert's product of such rows and weights, the rows
           quantised in the pass and the weights beforehand, as in serving

A case's "dir" is "fwd" (a serving or scoring call) or "step" (forward and
backward, as in training).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
BLOCK = 128


def listed():
    return [
        # the rows of one decode step: latency of the smallest calls
        {"name": "norm_decode", "op": "norm", "dir": "fwd", "T": 16, "D": 2048, "type": "bf16", "wtype": "bf16",
         "affine": True},
        # a training batch, its weights kept in 32 bits
        {"name": "norm_train", "op": "norm", "dir": "step", "T": 16384, "D": 4096, "type": "bf16", "wtype": "f32",
         "affine": True},
        # a small odd batch whose rows are no multiple of 16 bytes
        {"name": "norm_odd", "op": "norm", "dir": "step", "T": 1000, "D": 1001, "type": "f32", "wtype": "f32",
         "affine": True},
        # scoring a few tokens: the vocabulary's weights are read for a few rows
        {"name": "loss_score", "op": "loss", "dir": "fwd", "T": 8, "V": 32768, "D": 2048, "type": "bf16", "bias": False,
         "drop": 0.0},
        # evaluating a batch, every token's loss, a vocabulary of odd size
        {"name": "loss_eval", "op": "loss", "dir": "fwd", "T": 4096, "V": 50001, "D": 1024, "type": "f16", "bias": True,
         "drop": 0.1},
        # a training step over a large vocabulary: the largest case
        {"name": "loss_train", "op": "loss", "dir": "step", "T": 8192, "V": 65536, "D": 2048, "type": "bf16",
         "bias": False, "drop": 0.05},
        # small odd sizes in 32 bits
        {"name": "loss_odd", "op": "loss", "dir": "step", "T": 513, "V": 1001, "D": 257, "type": "f32", "bias": True,
         "drop": 0.2},
        # a decode step's rows to 8 bits and back
        {"name": "quant_decode", "op": "quant", "dir": "fwd", "T": 64, "D": 2048, "type": "bf16"},
        # an expert layer's weights to 8 bits when a model is loaded, and back to check them
        {"name": "quant_weights", "op": "quant", "dir": "fwd", "T": 65536, "D": 2048, "type": "bf16"},
        # a decode step's products: every chosen expert's weights are read for a few rows
        {"name": "linear8_decode", "op": "linear8", "dir": "fwd", "T": 16, "K": 2048, "F": 1024, "E": 64, "m": 4,
         "drop": 0.0, "idle": 0, "type": "bf16", "bias": True, "act": "silu"},
        # a prompt's products with many rows for each expert
        {"name": "linear8_prefill", "op": "linear8", "dir": "fwd", "T": 16384, "K": 2048, "F": 4096, "E": 8, "m": 2,
         "drop": 0.0, "idle": 0, "type": "bf16", "bias": True, "act": "silu"},
        # small odd layers, an expert without tokens
        {"name": "linear8_odd", "op": "linear8", "dir": "fwd", "T": 513, "K": 257, "F": 1001, "E": 7, "m": 2, "drop": 0.2,
         "idle": 1, "type": "f16", "bias": True, "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges: sizes spread over their
    logarithm, odd ones among them, every type and direction."""
    op = rng.choice(["norm", "norm", "loss", "loss", "loss", "quant", "linear8", "linear8"])
    # widths: multiples of 64, of 8, and any
    unit = rng.choice([64, 64, 8, 1])

    def width(lo, hi):
        return max(1, _log(rng, lo, hi) // unit) * unit

    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    c = {"op": op, "dir": rng.choice(["fwd", "step"]), "type": kind}
    if op == "norm":
        c |= {"D": width(64, 16384), "wtype": rng.choice([kind, "f32"]), "affine": rng.random() < 0.8}
        return c | {"T": _log(rng, 1, max(1, min(65536, (1 << 26) // c["D"])))}
    if op == "quant":
        c |= {"dir": "fwd", "D": width(64, 8192)}
        return c | {"T": _log(rng, 1, max(1, min(65536, (1 << 26) // c["D"])))}
    if op == "loss":
        c |= {"D": width(64, 4096), "V": _log(rng, 256, 65536), "bias": rng.random() < 0.5,
              "drop": rng.choice([0.0, 0.05, 0.3])}
        if rng.random() < 0.5:
            c["V"] = max(1, c["V"] // 64) * 64
        # 32-bit products run at a sixteenth of the 16-bit rate
        rows = (1 << 40 if kind != "f32" else 1 << 36) // (c["V"] * c["D"])
        return c | {"T": _log(rng, 1, max(1, min(8192, rows)))}
    E = _log(rng, 4, 128)
    m = rng.randint(1, min(8, E - 1))
    c |= {"dir": "fwd", "E": E, "m": m, "K": width(64, 4096), "F": width(64, 4096), "bias": rng.random() < 0.7,
          "drop": rng.choice([0.0, 0.05, 0.3]), "idle": rng.choice([0, 0, 1, 2]) if E - m > 2 else 0,
          "act": rng.choice(["none", "relu", "silu", "gelu"])}
    while E * c["K"] * c["F"] > 1 << 28:
        E = max(2, E // 2)
        c |= {"E": E, "m": min(m, E - 1), "idle": 0}
    pairs = (1 << 38) // (c["K"] * c["F"])
    return c | {"T": _log(rng, 1, max(1, min(32768, pairs) // c["m"]))}


# ---- blocks of 128 in 8 bits ---------------------------------------------------

def _two(e):
    """2^e in float32 for whole e in [-126, 127], exactly."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x):
    """(values, exponents): e4m3 values of x's rows in blocks of 128, padded
    with zeros to whole blocks, and each block's power of two: the least e with
    max|x| <= 448 2^e, 0 for a block of zeros."""
    pad = -x.shape[-1] % BLOCK
    x = torch.nn.functional.pad(x.float(), (0, pad))
    x = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = x.abs().amax(-1)
    part, e = torch.frexp(top)                     # top = part 2^e, part in [0.5, 1)
    e = torch.where(part <= 0.875, e - 9, e - 8).clamp(min=-127)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    q = (x * _two(-e)[..., None]).to(torch.float8_e4m3fn)
    return q.flatten(-2), e


def _dequantise(q, e, width):
    v = q.float().unflatten(-1, (-1, BLOCK))
    return (v * _two(e)[..., None]).flatten(-2)[..., :width]


# ---- inputs ----------------------------------------------------------------------

def _plan(case, gen):
    """Distinct experts of every token with uneven loads, idle ones never
    chosen, dropped slots empty: offsets, order and places of the pairs."""
    T, E, m = case["T"], case["E"], case["m"]
    load = torch.rand(E, generator=gen, device="cuda") + 0.5
    if case["idle"]:
        load[torch.randperm(E, generator=gen, device="cuda")[:case["idle"]]] = 0.0
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-9, 1 - 1e-7)))
    key = (load.log() + noise).topk(m, dim=1).indices.reshape(-1)
    if case["drop"]:
        key = torch.where(torch.rand(T * m, generator=gen, device="cuda") < case["drop"], E, key)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    pos = torch.arange(T * m, device="cuda")
    place = torch.empty_like(order)
    place[order] = pos
    place = torch.where(key == E, -1, place).reshape(T, m)
    order = torch.where(pos < offsets[-1], order, -1)
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = DTYPES[case["type"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale)

    s = {"case": case}
    if case["op"] in ("norm", "quant"):
        T, D = case["T"], case["D"]
        # rows of different sizes, as a residual stream has them
        size = torch.exp(normal(T, 1, scale=0.5))
        s["x"] = (normal(T, D) * size + (0.5 * size if case["op"] == "norm" else 0)).to(kind)
        if case["op"] == "norm":
            w = DTYPES[case["wtype"]]
            s["weight"] = (1 + normal(D, scale=0.2)).to(w) if case["affine"] else None
            s["bias"] = normal(D, scale=0.2).to(w) if case["affine"] else None
            s["dy"] = normal(T, D).to(kind)
        return s
    if case["op"] == "loss":
        T, V, D = case["T"], case["V"], case["D"]
        s["x"] = normal(T, D).to(kind)
        s["weight"] = normal(V, D, scale=2 * D ** -0.5).to(kind)
        s["bias"] = normal(V, scale=0.5).to(kind) if case["bias"] else None
        s["target"] = torch.randint(V, (T,), generator=gen, device="cuda")
        if case["drop"]:  # padding and prompts
            s["target"][torch.rand(T, generator=gen, device="cuda") < case["drop"]] = -100
        # 16-bit gradients of fp16 are scaled, as loss scaling does
        s["dloss"] = torch.rand((), generator=gen, device="cuda") + (4096.0 if case["type"] == "f16" else 0.5)
        return s
    K, F, E = case["K"], case["F"], case["E"]
    s["offsets"], s["order"], s["place"] = _plan(case, gen)
    s["xs"] = normal(case["T"] * case["m"], K).to(kind)
    s["xs"][int(s["offsets"][-1]):] = 0  # as dispatch leaves the unused places
    w = [_quantise(normal(F, K, scale=K ** -0.5).to(kind)) for _ in range(E)]
    s["weight"] = torch.stack([q.view(torch.uint8) for q, _ in w]).view(torch.float8_e4m3fn)
    s["scales"] = torch.stack([e + 127 for _, e in w]).to(torch.uint8).view(torch.float8_e8m0fnu)
    s["bias"] = normal(E, F, scale=0.5).to(kind) if case["bias"] else None
    # the row capacity the plain form pads every expert to
    s["cap"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    return s


# ---- plain forms -------------------------------------------------------------------

def _plain_norm(s):
    x, kind = s["x"].float(), s["x"].dtype
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
    xh = (x - mean) * rstd
    w = s["weight"]
    y = (xh * w.float() + s["bias"].float() if w is not None else xh).to(kind)
    if s["case"]["dir"] == "fwd":
        return y
    dy = s["dy"].float()
    g = dy * w.float() if w is not None else dy
    dx = (rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))).to(kind)
    if w is None:
        return y, dx
    return y, dx, (dy * xh).sum(0).to(w.dtype), dy.sum(0).to(w.dtype)


def _plain_loss(s):
    x, w, target = s["x"].float(), s["weight"].float(), s["target"]
    T, V = x.shape[0], w.shape[0]
    z = x @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    top = z.amax(1, keepdim=True)
    lse = (z - top).exp().sum(1, keepdim=True).log() + top
    on = (target >= 0) & (target < V)
    at = target.clamp(0, V - 1)[:, None]
    loss = torch.where(on, (lse - z.gather(1, at))[:, 0], torch.zeros((), device="cuda"))
    if s["case"]["dir"] == "fwd":
        return loss
    count = on.sum().clamp(min=1)
    g = on * (s["dloss"] / count)
    d = (z - lse).exp() * g[:, None]
    d.scatter_add_(1, at, -g[:, None])
    dx, dw = (d @ w).to(s["x"].dtype), (d.t() @ x).to(s["x"].dtype)
    out = (loss.sum() / count, dx, dw)
    return out + (d.sum(0).to(s["x"].dtype),) if s["bias"] is not None else out


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _plain_linear8(s):
    """One batched product over the experts, their rows padded to one length."""
    case = s["case"]
    K, off = case["K"], s["offsets"].long()
    x = _dequantise(*_quantise(s["xs"]), K)
    weight = _dequantise(s["weight"], s["scales"].view(torch.uint8).int() - 127, K)
    row = off[:-1, None] + torch.arange(max(1, s["cap"]), device="cuda")[None, :]
    on = row < off[1:, None]
    x = x[row.clamp(max=x.shape[0] - 1)] * on[:, :, None]
    z = torch.bmm(x, weight.transpose(1, 2).contiguous())
    if s["bias"] is not None:
        z = z + s["bias"].float()[:, None, :]
    y = torch.zeros(s["xs"].shape[0], case["F"], dtype=s["xs"].dtype, device="cuda")
    y[row[on]] = _act(z, case["act"]).to(s["xs"].dtype)[on]
    return y


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "loss":
        return _plain_loss(s)
    if op == "quant":
        return _dequantise(*_quantise(s["x"]), s["case"]["D"]).to(s["x"].dtype)
    return _plain_linear8(s)


# ---- the package's operators ---------------------------------------------------------

def _own(s):
    import differentiable_exact_budget_amd as L

    case = s["case"]
    op, step = case["op"], case["dir"] == "step"
    if op == "quant":
        return L.expert_dequantize(L.expert_quantize(s["x"]), s["x"].dtype)
    if op == "linear8":
        plan = L.ExpertPlan(case["E"], s["offsets"], s["order"], s["place"])
        weight = L.ScaledRows(s["weight"], s["scales"], case["K"])
        return L.expert_linear_fp8(L.expert_quantize(s["xs"]), weight, plan, bias=s["bias"], activation=case["act"],
                                   dtype=s["xs"].dtype)
    names = ("x", "weight", "bias")
    given = {k: s[k].detach().requires_grad_(step) for k in names if s[k] is not None}
    leaves = list(given.values())
    if op == "norm":
        y = L.layer_norm(given["x"], given.get("weight"), given.get("bias"), eps=EPS)
        return (y.detach(), *torch.autograd.grad(y, leaves, s["dy"])) if step else y
    loss = L.linear_cross_entropy(given["x"], given["weight"], s["target"], bias=given.get("bias"),
                                  reduction="mean" if step else "none")
    return (loss.detach(), *torch.autograd.grad(loss, leaves, s["dloss"])) if step else loss


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -----------------------------------------------------

def work(case):
    op, T, step = case["op"], case["T"], case["dir"] == "step"
    size = 4 if case["type"] == "f32" else 2
    if op == "norm":
        n, w = T * case["D"], (4 if case["wtype"] == "f32" else 2) * case["D"] if case["affine"] else 0
        return {"bytes": 2 * n * size + 2 * w + (3 * n * size + 3 * w if step else 0),
                "flops": (8 + (14 if step else 0)) * n}
    if op == "quant":
        n = T * case["D"]
        return {"bytes": 2 * n * size, "flops": 4 * n}
    if op == "loss":
        V, D = case["V"], case["D"]
        n = (T + V) * D * size + (V * size if case["bias"] else 0)
        return {"bytes": n * (2 if step else 1) + 8 * T + (4 if step else 4 * T),
                "flops": (6 if step else 2) * T * V * D}
    K, F, E, m = case["K"], case["F"], case["E"], case["m"]
    live = T * m * (1 - case["drop"])
    busy = max(1, E - case["idle"])
    active = busy * (1 - (1 - min(1.0, m * (1 - case["drop"]) / busy)) ** T)
    b = active * F * (K * (1 + 1 / BLOCK) + (size if case["bias"] else 0)) + live * K * size + T * m * F * size
    return {"bytes": b, "flops": 2 * live * K * F}


# ---- the definition in 64 bits -----------------------------------------------------------

def _grid(x):
    """What blocks of 128 in 8 bits stand for, as numbers: each to the nearest
    of the e4m3 grid under its block's power of two, ties to even."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[-1], BLOCK):
        v = x[..., c:c + BLOCK].double()
        top = v.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
        # the logarithm may be off next to a whole number
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where((top > 0) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e).clamp(min=-127.0)
        u = v / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
        out[..., c:c + BLOCK] = torch.round(u / step) * step * torch.exp2(e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, step = case["op"], case["dir"] == "step"
    if op == "quant":
        return _grid(s["x"])
    if op == "norm":
        x = s["x"].double()
        n = x.shape[1]
        mu = x.sum(1, keepdim=True) / n
        sd = torch.sqrt((x * x).sum(1, keepdim=True) / n - mu * mu + EPS)
        w = s["weight"].double() if case["affine"] else torch.ones(n, dtype=torch.float64, device="cuda")
        y = (x - mu) / sd * w + (s["bias"].double() if case["affine"] else 0)
        if not step:
            return y
        dy = s["dy"].double()
        a = dy * w
        # y's row Jacobian: (delta_ij - 1/n - (x_i - mu)(x_j - mu) / (n sd^2)) / sd
        dot = (a * (x - mu)).sum(1, keepdim=True)
        dx = (a - a.sum(1, keepdim=True) / n - (x - mu) * dot / (n * sd * sd)) / sd
        if not case["affine"]:
            return y, dx
        return y, dx, (dy * (x - mu) / sd).sum(0), dy.sum(0)
    if op == "loss":
        x, w = s["x"].double(), s["weight"].double()
        T, V = x.shape[0], w.shape[0]
        count = max(1, int(((s["target"] >= 0) & (s["target"] < V)).sum()))
        losses = torch.zeros(T, dtype=torch.float64, device="cuda")
        dx = torch.zeros_like(x)
        dw = torch.zeros_like(w)
        db = torch.zeros(V, dtype=torch.float64, device="cuda")
        for t in range(0, T, 2048):
            z = torch.addmm(s["bias"].double(), x[t:t + 2048], w.t()) if case["bias"] else x[t:t + 2048] @ w.t()
            y = s["target"][t:t + 2048]
            live = ((y >= 0) & (y < V)).nonzero()[:, 0]
            logp = torch.log_softmax(z[live], 1)
            losses[t + live] = -logp[torch.arange(live.numel(), device="cuda"), y[live]]
            if step:
                d = torch.exp(logp)
                d[torch.arange(live.numel(), device="cuda"), y[live]] -= 1
                d *= s["dloss"].double() / count
                dx[t + live] = d @ w
                dw += d.t() @ x[t + live]
                db += d.sum(0)
        if not step:
            return losses
        out = (losses.sum() / count, dx, dw)
        return out + (db,) if case["bias"] else out
    off = s["offsets"].tolist()
    x = _grid(s["xs"])
    y = torch.zeros(x.shape[0], case["F"], dtype=torch.float64, device="cuda")
    scale = torch.exp2(s["scales"].view(torch.uint8).double() - 127)
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        w = (s["weight"][e].double() * scale[e].repeat_interleave(BLOCK, 1))[:, :case["K"]]
        z = x[a:b] @ w.t()
        if case["bias"]:
            z = z + s["bias"][e].double()
        y[a:b] = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z / (1 + torch.exp(-z)),
                  "gelu": lambda: z * 0.5 * (1 + torch.erf(z / math.sqrt(2.0)))}[case["act"]]()
    return y
