"""Routed experts on MI355X: from exact-budget gates to the experts' outputs.

    p = soft_topk_rows(scores, k, t)                  # gates, each row sums to k
    ids, w = expert_topk(p, m, normalize=True)        # the m largest of every row
    plan = expert_sort(ids, experts)                  # pairs in expert order
    xs = expert_dispatch(x, plan)                     # rows to their places
    ys = expert_linear(xs, weight, plan, bias=bias, activation="silu")
    out = expert_combine(ys, w, plan, residual=x)     # weighted rows back

All of them but the sort are differentiable; each gradient also has an entry
point of its own (expert_*_vjp).  They run in liblapsum.so (hand-written HIP
for gfx950, the C ABI of include/lapsum_experts.h) on the caller's current
stream, never wait for the device and can be captured into a graph: the number
of pairs in use stays on the device, and every array that goes by positions
has tokens * slots rows, zeros past plan.offsets[experts].

Rows may be float32, bfloat16 or float16; gates and weights are float32.
Sums are held in float32 and rounded once to the rows' type.
"""
import ctypes

import torch

from . import _binding
from ._binding import LapsumError

__all__ = ["ExpertPlan", "expert_topk", "expert_topk_vjp", "expert_sort", "expert_dispatch", "expert_dispatch_vjp",
           "expert_linear", "expert_linear_vjp", "expert_combine", "expert_combine_vjp", "ACTIVATIONS",
           "MAX_EXPERTS", "MAX_SLOTS"]

MAX_EXPERTS, MAX_SLOTS = 1024, 64
ACTIVATIONS = ("none", "relu", "silu", "gelu")
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

EXPORTED = [
    "lapsum_expert_topk", "lapsum_expert_topk_vjp", "lapsum_expert_sort_scratch_bytes", "lapsum_expert_sort",
    "lapsum_expert_dispatch", "lapsum_expert_dispatch_vjp", "lapsum_expert_combine", "lapsum_expert_combine_vjp",
    "lapsum_expert_linear", "lapsum_expert_linear_vjp_scratch_bytes", "lapsum_expert_linear_vjp",
]

_lib = None


def lib():
    """liblapsum.so with the expert operators' argument types set.  These
    calls only launch, so they keep the interpreter lock (PyDLL): giving it up
    and taking it again costs more than the call."""
    global _lib
    if _lib is None:
        _binding.lib()  # raises if it is not built
        L = ctypes.PyDLL(_binding.LIB_PATH)
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        types = {
            "lapsum_expert_topk": [vp, i64, i64, i64, f32, i32, vp, vp, vp, vp],
            "lapsum_expert_topk_vjp": [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp],
            "lapsum_expert_sort_scratch_bytes": [i64, i64],
            "lapsum_expert_sort": [vp, i64, i64, vp, vp, vp, vp, vp],
            "lapsum_expert_dispatch": [vp, i32, i64, i64, i64, i64, vp, vp, vp, vp],
            "lapsum_expert_dispatch_vjp": [vp, i32, i64, i64, i64, vp, vp, vp],
            "lapsum_expert_combine": [vp, vp, vp, i32, i64, i64, i64, vp, vp, vp],
            "lapsum_expert_combine_vjp": [vp, vp, vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, vp],
            "lapsum_expert_linear": [vp, vp, vp, i32, i64, i64, i64, i64, vp, i32, vp, vp, vp],
            "lapsum_expert_linear_vjp_scratch_bytes": [i32, i64, i64, i64, i64, i32, i32],
            "lapsum_expert_linear_vjp": [vp, vp, vp, vp, i32, i64, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp],
        }
        for name, args in types.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_size_t if name.endswith("_bytes") else ctypes.c_int
        _lib = L
    return _lib


def _check(x, name: str, dtypes, dims: int, device=None) -> None:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device (got {x.device})")
    if device is not None and x.device != device:
        raise ValueError(f"{name} must be on {device} (got {x.device})")
    if x.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)} (got {x.dtype})")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions (got {x.dim()})")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(x, name: str, shape) -> None:
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)} (got {tuple(x.shape)})")


def _ptr(x):
    return None if x is None else x.data_ptr()


def _recorded(*inputs) -> bool:
    """Whether autograd has to see the call."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)


def _any_rows(*outputs) -> bool:
    """Whether any output is wanted and has elements to write."""
    return any(t is not None and t.numel() for t in outputs)


def _run(name: str, device, *args) -> None:
    """Calls the C entry point on the device's current stream."""
    f, i = getattr(_lib or lib(), name), device.index
    if i == torch.cuda.current_device():
        rc = f(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            rc = f(*args, torch._C._cuda_getCurrentRawStream(i))
    if rc != 0:
        raise LapsumError(rc, name)


class ExpertPlan:
    """Where every (token, slot) pair goes, as expert_sort makes it.

    offsets[e] .. offsets[e + 1] - 1 are the positions of expert e's pairs and
    offsets[experts] is the number of pairs in use; order[pos] is the pair
    token * slots + slot at a position (-1 past the used ones), place[token,
    slot] the position of a pair (-1 for an empty slot).  All int32."""
    __slots__ = ("experts", "offsets", "order", "place")

    def __init__(self, experts: int, offsets: torch.Tensor, order: torch.Tensor, place: torch.Tensor):
        self.experts, self.offsets, self.order, self.place = experts, offsets, order, place

    @property
    def tokens(self) -> int:
        return self.place.shape[0]

    @property
    def slots(self) -> int:
        return self.place.shape[1]

    def check(self, device) -> None:
        """Raises where the arrays do not fit one another (their values are
        only bounds-checked, on the device)."""
        _check(self.offsets, "plan.offsets", (torch.int32,), 1, device)
        _check(self.order, "plan.order", (torch.int32,), 1, device)
        _check(self.place, "plan.place", (torch.int32,), 2, device)
        _shape(self.offsets, "plan.offsets", (self.experts + 1,))
        _shape(self.order, "plan.order", (self.place.numel(),))


def _check_plan(plan, device) -> None:
    if not isinstance(plan, ExpertPlan):
        raise TypeError("plan must be an ExpertPlan")
    plan.check(device)


# ---- the m largest gates ------------------------------------------------------

def _topk(p: torch.Tensor, m: int, floor: float, normalize: bool):
    _check(p, "p", (torch.float32,), 2)
    tokens, experts = p.shape
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"p must have between 1 and {MAX_EXPERTS} experts (got {experts})")
    if not 1 <= m <= min(experts, MAX_SLOTS):
        raise ValueError(f"m must be between 1 and min(experts, {MAX_SLOTS}) (got {m})")
    if floor != floor:
        raise ValueError("floor must not be NaN")
    ids = torch.empty(tokens, m, dtype=torch.int32, device=p.device)
    w = torch.empty(tokens, m, dtype=torch.float32, device=p.device)
    sums = torch.empty(tokens, dtype=torch.float32, device=p.device) if normalize else None
    _run("lapsum_expert_topk", p.device, p.data_ptr(), tokens, experts, m, floor, int(normalize), ids.data_ptr(),
         w.data_ptr(), _ptr(sums))
    return ids, w, sums


def expert_topk_vjp(ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor, experts: int,
                    sums: torch.Tensor = None) -> torch.Tensor:
    """dp [tokens, experts] of expert_topk from dw; sums (the rows' sums of
    chosen gates) where the weights were normalized, else None."""
    _check(ids, "ids", (torch.int32,), 2)
    for name, x in (("w", w), ("dw", dw)):
        _check(x, name, (torch.float32,), 2, ids.device)
        _shape(x, name, ids.shape)
    tokens, m = ids.shape
    if sums is not None:
        _check(sums, "sums", (torch.float32,), 1, ids.device)
        _shape(sums, "sums", (tokens,))
    dp = torch.empty(tokens, experts, dtype=torch.float32, device=ids.device)
    _run("lapsum_expert_topk_vjp", ids.device, ids.data_ptr(), w.data_ptr(), dw.data_ptr(), _ptr(sums), tokens,
         experts, m, int(sums is not None), dp.data_ptr())
    return dp


class ExpertTopK(torch.autograd.Function):
    """The choice of the m largest gates; backward scatters to the chosen."""

    @staticmethod
    def forward(ctx, p, m, floor, normalize):
        ids, w, sums = _topk(p.contiguous(), m, floor, normalize)
        ctx.save_for_backward(ids, w, sums)
        ctx.experts = p.shape[1]
        ctx.mark_non_differentiable(ids)
        ctx.set_materialize_grads(False)
        return ids, w

    @staticmethod
    def backward(ctx, _, dw):
        if dw is None:
            return None, None, None, None
        ids, w, sums = ctx.saved_tensors
        dp = expert_topk_vjp(ids, w, dw.contiguous().to(torch.float32), ctx.experts, sums)
        return dp, None, None, None


def expert_topk(p: torch.Tensor, m: int, *, floor: float = float("-inf"), normalize: bool = False):
    """(ids, w), int32 and float32 [tokens, m]: the m largest gates of every
    row of p [tokens, experts] in descending order, ties to the lowest expert.

    A gate is chosen only when it is greater than `floor` (NaN and -inf never
    are); slots left over have id -1 and weight 0.  With `normalize` the
    weights are divided by their row's sum (all 0 where it is not above 0).
    Differentiable with respect to p through w."""
    if not isinstance(p, torch.Tensor):
        raise TypeError("p must be a torch.Tensor")
    if not _recorded(p):
        return _topk(p.contiguous(), int(m), float(floor), bool(normalize))[:2]
    return ExpertTopK.apply(p, int(m), float(floor), bool(normalize))


# ---- pairs in expert order ----------------------------------------------------

def expert_sort(ids: torch.Tensor, experts: int) -> ExpertPlan:
    """The plan of ids [tokens, slots] (int32; an id outside [0, experts) is
    an empty slot): a stable counting sort of the pairs by expert."""
    _check(ids, "ids", (torch.int32,), 2)
    tokens, slots = ids.shape
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"experts must be between 1 and {MAX_EXPERTS} (got {experts})")
    if not 1 <= slots <= MAX_SLOTS:
        raise ValueError(f"ids must have between 1 and {MAX_SLOTS} slots (got {slots})")
    dev, pairs = ids.device, tokens * slots
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    order = torch.empty(pairs, dtype=torch.int32, device=dev)
    place = torch.empty(tokens, slots, dtype=torch.int32, device=dev)
    n = lib().lapsum_expert_sort_scratch_bytes(pairs, experts)
    scratch = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    _run("lapsum_expert_sort", dev, ids.data_ptr(), pairs, experts, offsets.data_ptr(), order.data_ptr(),
         place.data_ptr(), _ptr(scratch))
    return ExpertPlan(experts, offsets, order, place)


# ---- rows to their places -----------------------------------------------------

def _dispatch(x: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    _check(x, "x", _DTYPES, 2)
    _check_plan(plan, x.device)
    _shape(x, "x", (plan.tokens, x.shape[1]))
    xs = torch.empty(plan.tokens * plan.slots, x.shape[1], dtype=x.dtype, device=x.device)
    _run("lapsum_expert_dispatch", x.device, x.data_ptr(), _DTYPES[x.dtype], plan.tokens, plan.slots, x.shape[1],
         plan.experts, plan.offsets.data_ptr(), plan.place.data_ptr(), xs.data_ptr())
    return xs


def expert_dispatch_vjp(dxs: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """dx[token] = the sum of the token's rows of dxs, in slot order."""
    _check(dxs, "dxs", _DTYPES, 2)
    _check_plan(plan, dxs.device)
    _shape(dxs, "dxs", (plan.tokens * plan.slots, dxs.shape[1]))
    dx = torch.empty(plan.tokens, dxs.shape[1], dtype=dxs.dtype, device=dxs.device)
    _run("lapsum_expert_dispatch_vjp", dxs.device, dxs.data_ptr(), _DTYPES[dxs.dtype], plan.tokens, plan.slots,
         dxs.shape[1], plan.place.data_ptr(), dx.data_ptr())
    return dx


class ExpertDispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return _dispatch(x.contiguous(), plan)

    @staticmethod
    def backward(ctx, dxs):
        return expert_dispatch_vjp(dxs.contiguous(), ctx.plan), None


def expert_dispatch(x: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """xs [tokens * slots, width]: every pair's row of x [tokens, width] at
    the pair's place, zeros past the used places."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not _recorded(x):
        return _dispatch(x.contiguous(), plan)
    return ExpertDispatch.apply(x, plan)


# ---- the experts' products ----------------------------------------------------

def _linear_shapes(xs, weight, plan, bias, activation):
    _check(xs, "xs", _DTYPES, 2)
    _check(weight, "weight", (xs.dtype,), 3, xs.device)
    _check_plan(plan, xs.device)
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)} (got {activation!r})")
    experts, out, width = weight.shape
    _shape(xs, "xs", (plan.tokens * plan.slots, width))
    _shape(weight, "weight", (plan.experts, out, width))
    if bias is not None:
        _check(bias, "bias", (xs.dtype,), 2, xs.device)
        _shape(bias, "bias", (experts, out))
    return xs.shape[0], width, out, experts


def _linear(xs, weight, plan, bias, activation, keep):
    rows, width, out, experts = _linear_shapes(xs, weight, plan, bias, activation)
    ys = torch.empty(rows, out, dtype=xs.dtype, device=xs.device)
    z = None
    if keep and activation != "none":
        z = torch.empty(rows, out, dtype=torch.float32 if xs.dtype == torch.float32 else torch.float16,
                        device=xs.device)
    _run("lapsum_expert_linear", xs.device, xs.data_ptr(), weight.data_ptr(), _ptr(bias), _DTYPES[xs.dtype], rows,
         width, out, experts, plan.offsets.data_ptr(), ACTIVATIONS.index(activation), ys.data_ptr(), _ptr(z))
    return ys, z


def expert_linear_vjp(xs: torch.Tensor, weight: torch.Tensor, plan: ExpertPlan, z: torch.Tensor, dys: torch.Tensor, *,
                      activation: str = "none", want=(True, True, True)):
    """(dxs, dweight, dbias) of expert_linear; `want` leaves out (None) those
    that are not needed.  z is what the forward kept (None without an
    activation): float32 for float32 rows, else float16."""
    rows, width, out, experts = _linear_shapes(xs, weight, plan, None, activation)
    _check(dys, "dys", (xs.dtype,), 2, xs.device)
    _shape(dys, "dys", (rows, out))
    if activation != "none":
        _check(z, "z", (torch.float32 if xs.dtype == torch.float32 else torch.float16,), 2, xs.device)
        _shape(z, "z", (rows, out))
    dxs = torch.empty_like(xs) if want[0] else None
    dweight = torch.empty_like(weight) if want[1] else None
    dbias = torch.empty(experts, out, dtype=xs.dtype, device=xs.device) if want[2] else None
    if not _any_rows(dxs, dweight, dbias):
        return dxs, dweight, dbias
    act, dt = ACTIVATIONS.index(activation), _DTYPES[xs.dtype]
    n = lib().lapsum_expert_linear_vjp_scratch_bytes(dt, rows, width, out, experts, act, int(bool(want[2])))
    scratch = torch.empty(n, dtype=torch.uint8, device=xs.device) if n else None
    _run("lapsum_expert_linear_vjp", xs.device, xs.data_ptr(), weight.data_ptr(), _ptr(z), dys.data_ptr(), dt, rows,
         width, out, experts, plan.offsets.data_ptr(), act, _ptr(dxs), _ptr(dweight), _ptr(dbias), _ptr(scratch))
    return dxs, dweight, dbias


class ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, xs, weight, bias, plan, activation):
        xs, weight = xs.contiguous(), weight.contiguous()
        keep = any(ctx.needs_input_grad)
        ys, z = _linear(xs, weight, plan, bias.contiguous() if bias is not None else None, activation, keep)
        if keep:
            ctx.save_for_backward(xs, weight, z)
            ctx.plan, ctx.activation = plan, activation
        return ys

    @staticmethod
    def backward(ctx, dys):
        xs, weight, z = ctx.saved_tensors
        dxs, dweight, dbias = expert_linear_vjp(xs, weight, ctx.plan, z, dys.contiguous(), activation=ctx.activation,
                                                want=ctx.needs_input_grad[:3])
        return dxs, dweight, dbias, None, None


def expert_linear(xs: torch.Tensor, weight: torch.Tensor, plan: ExpertPlan, *, bias: torch.Tensor = None,
                  activation: str = "none") -> torch.Tensor:
    """ys [rows, out]: act(xs W_e^T + b_e), e the expert of each row by the
    plan; zeros past the used rows.  weight [experts, out, in], bias [experts,
    out] or None, all of one dtype; activation "none", "relu", "silu" or
    "gelu" (the exact one, with the error function)."""
    if not isinstance(xs, torch.Tensor) or not isinstance(weight, torch.Tensor):
        raise TypeError("xs and weight must be torch.Tensors")
    if not _recorded(xs, weight, bias):
        return _linear(xs.contiguous(), weight.contiguous(), plan, bias.contiguous() if bias is not None else None,
                       activation, False)[0]
    return ExpertLinear.apply(xs, weight, bias, plan, activation)


# ---- weighted rows back -------------------------------------------------------

def _combine_shapes(ys, w, plan):
    _check(ys, "ys", _DTYPES, 2)
    _check_plan(plan, ys.device)
    _shape(ys, "ys", (plan.tokens * plan.slots, ys.shape[1]))
    _check(w, "w", (torch.float32,), 2, ys.device)
    _shape(w, "w", (plan.tokens, plan.slots))
    return ys.shape[1]


def _combine(ys, w, plan, residual):
    width = _combine_shapes(ys, w, plan)
    if residual is not None:
        _check(residual, "residual", (ys.dtype,), 2, ys.device)
        _shape(residual, "residual", (plan.tokens, width))
    out = torch.empty(plan.tokens, width, dtype=ys.dtype, device=ys.device)
    _run("lapsum_expert_combine", ys.device, ys.data_ptr(), w.data_ptr(), _ptr(residual), _DTYPES[ys.dtype],
         plan.tokens, plan.slots, width, plan.place.data_ptr(), out.data_ptr())
    return out


def expert_combine_vjp(ys: torch.Tensor, w: torch.Tensor, plan: ExpertPlan, dout: torch.Tensor, *,
                       want=(True, True)):
    """(dys, dw) of expert_combine; `want` leaves out (None) what is not needed."""
    width = _combine_shapes(ys, w, plan)
    _check(dout, "dout", (ys.dtype,), 2, ys.device)
    _shape(dout, "dout", (plan.tokens, width))
    dys = torch.empty_like(ys) if want[0] else None
    dw = torch.empty_like(w) if want[1] else None
    if not _any_rows(dys, dw):
        return dys, dw
    _run("lapsum_expert_combine_vjp", ys.device, ys.data_ptr(), w.data_ptr(), dout.data_ptr(), _DTYPES[ys.dtype],
         plan.tokens, plan.slots, width, plan.experts, plan.offsets.data_ptr(), plan.place.data_ptr(), _ptr(dys),
         _ptr(dw))
    return dys, dw


class ExpertCombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, w, residual, plan):
        ys, w = ys.contiguous(), w.contiguous()
        ctx.save_for_backward(ys, w)
        ctx.plan = plan
        return _combine(ys, w, plan, residual.contiguous() if residual is not None else None)

    @staticmethod
    def backward(ctx, dout):
        ys, w = ctx.saved_tensors
        dys, dw = expert_combine_vjp(ys, w, ctx.plan, dout.contiguous(), want=ctx.needs_input_grad[:2])
        return dys, dw, dout if ctx.needs_input_grad[2] else None, None


def expert_combine(ys: torch.Tensor, w: torch.Tensor, plan: ExpertPlan, *,
                   residual: torch.Tensor = None) -> torch.Tensor:
    """out [tokens, width]: residual + the sum over a token's slots of
    w[token, slot] times the slot's row of ys; empty slots add nothing."""
    if not isinstance(ys, torch.Tensor) or not isinstance(w, torch.Tensor):
        raise TypeError("ys and w must be torch.Tensors")
    if not _recorded(ys, w, residual):
        return _combine(ys.contiguous(), w.contiguous(), plan, residual.contiguous() if residual is not None else None)
    return ExpertCombine.apply(ys, w, residual, plan)
