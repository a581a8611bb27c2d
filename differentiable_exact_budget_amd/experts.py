"""Routed experts on MI355X: from exact-budget gates to the experts' outputs.

    p = soft_topk_rows(scores, k, t)                  # gates, each row sums to k
    ids, w = expert_topk(p, m, normalize=True)        # the m largest of every row
    plan = expert_sort(ids, experts)                  # pairs in expert order
    xs = expert_dispatch(x, plan)                     # rows to their places
    ys = expert_linear(xs, weight, plan, bias=bias, activation="silu")
    out = expert_combine(ys, w, plan, residual=x)     # weighted rows back

All of them but the sort are differentiable, once and in reverse mode (second
derivatives and forward-mode tangents are refused, and so is torch.jit.trace);
each gradient also has an entry point of its own (expert_*_vjp).  They run in liblapsum.so (hand-written HIP
for gfx950, the C ABI of include/lapsum_experts.h) on the caller's current
stream, never wait for the device and can be captured into a graph: the number
of pairs in use stays on the device, and every array that goes by positions
has tokens * slots rows, zeros past plan.offsets[experts].

Rows may be float32, bfloat16 or float16; gates and weights are float32.
Sums are held in float32 and rounded once to the rows' type.
"""
import ctypes
import os

import torch

from . import _binding

__all__ = ["ExpertPlan", "expert_topk", "expert_topk_vjp", "expert_sort", "expert_dispatch", "expert_dispatch_vjp",
           "expert_linear", "expert_linear_forward", "expert_linear_vjp", "expert_combine", "expert_combine_vjp",
           "ACTIVATIONS", "MAX_EXPERTS", "MAX_SLOTS"]

MAX_EXPERTS, MAX_SLOTS = 1024, 64
ACTIVATIONS = ("none", "relu", "silu", "gelu")

EXPORTED = [
    "lapsum_expert_topk", "lapsum_expert_topk_vjp", "lapsum_expert_sort_scratch_bytes", "lapsum_expert_sort",
    "lapsum_expert_dispatch", "lapsum_expert_dispatch_vjp", "lapsum_expert_combine", "lapsum_expert_combine_vjp",
    "lapsum_expert_linear", "lapsum_expert_linear_vjp_scratch_bytes", "lapsum_expert_linear_vjp",
]

_lib = None
_torch_module = None


def lib():
    """ctypes view of the operators' C ABI in liblapsum.so."""
    global _lib
    if _lib is None:
        L = _binding.lib()
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


def _native():
    """The torch module over that ABI; raise if it has not been built."""
    global _torch_module
    if _torch_module is None:
        _binding.lib()  # loads liblapsum.so, or says that it is missing
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_experts_torch.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first "
                               "(python -c 'import __graft_entry__; __graft_entry__.build()')")
        from . import _experts_torch
        _torch_module = _experts_torch
    return _torch_module


def _tensors(**named) -> None:
    for name, x in named.items():
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


class ExpertPlan:
    """Where every (token, slot) pair goes, as expert_sort makes it.

    offsets[e] .. offsets[e + 1] - 1 are the positions of expert e's pairs and
    offsets[experts] is the number of pairs in use; order[pos] is the pair
    token * slots + slot at a position (-1 past the used ones), place[token,
    slot] the position of a pair (-1 for an empty slot).  All int32.  The
    operators check that the arrays fit one another; their values are only
    bounds-checked, on the device."""
    __slots__ = ("experts", "offsets", "order", "place")

    def __init__(self, experts: int, offsets: torch.Tensor, order: torch.Tensor, place: torch.Tensor):
        self.experts, self.offsets, self.order, self.place = experts, offsets, order, place

    @property
    def tokens(self) -> int:
        return self.place.shape[0]

    @property
    def slots(self) -> int:
        return self.place.shape[1]


def _arrays(plan):
    if not isinstance(plan, ExpertPlan):
        raise TypeError("plan must be an ExpertPlan")
    return plan.experts, plan.offsets, plan.order, plan.place


def expert_topk(p: torch.Tensor, m: int, *, floor: float = float("-inf"), normalize: bool = False):
    """(ids, w), int32 and float32 [tokens, m]: the m largest gates of every
    row of p [tokens, experts] in descending order, ties to the lowest expert.

    A gate is chosen only when it is greater than `floor` (NaN and -inf never
    are); slots left over have id -1 and weight 0.  With `normalize` the
    weights are divided by their row's sum (all 0 where it is not above 0).
    Differentiable with respect to p through w."""
    _tensors(p=p)
    return (_torch_module or _native()).topk(p, m, floor, normalize)


def expert_topk_vjp(ids: torch.Tensor, w: torch.Tensor, dw: torch.Tensor, experts: int,
                    sums: torch.Tensor = None) -> torch.Tensor:
    """dp [tokens, experts] of expert_topk from dw; sums (the rows' sums of
    chosen gates) where the weights were normalized, else None."""
    _tensors(ids=ids, w=w, dw=dw)
    return _native().topk_vjp(ids, w, dw, experts, sums)


def expert_sort(ids: torch.Tensor, experts: int) -> ExpertPlan:
    """The plan of ids [tokens, slots] (int32; an id outside [0, experts) is
    an empty slot): a stable counting sort of the pairs by expert."""
    _tensors(ids=ids)
    return ExpertPlan(experts, *(_torch_module or _native()).sort(ids, experts))


def expert_dispatch(x: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """xs [tokens * slots, width]: every pair's row of x [tokens, width] at
    the pair's place, zeros past the used places."""
    _tensors(x=x)
    return (_torch_module or _native()).dispatch(x, *_arrays(plan))


def expert_dispatch_vjp(dxs: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """dx[token] = the sum of the token's rows of dxs, in slot order."""
    _tensors(dxs=dxs)
    return _native().dispatch_vjp(dxs, *_arrays(plan))


def expert_linear(xs: torch.Tensor, weight: torch.Tensor, plan: ExpertPlan, *, bias: torch.Tensor = None,
                  activation: str = "none") -> torch.Tensor:
    """ys [rows, out]: act(xs W_e^T + b_e), e the expert of each row by the
    plan; zeros past the used rows.  weight [experts, out, in], bias [experts,
    out] or None, all of one dtype; activation "none", "relu", "silu" or
    "gelu" (the exact one, with the error function)."""
    _tensors(xs=xs, weight=weight)
    return (_torch_module or _native()).linear(xs, weight, bias, activation, *_arrays(plan))


def expert_linear_forward(xs: torch.Tensor, weight: torch.Tensor, plan: ExpertPlan, *, bias: torch.Tensor = None,
                          activation: str = "none"):
    """(ys, z) of expert_linear, outside autograd: z is what
    expert_linear_vjp wants of the forward pass (None without an activation)."""
    _tensors(xs=xs, weight=weight)
    return _native().linear_forward(xs, weight, bias, activation, *_arrays(plan))


def expert_linear_vjp(xs: torch.Tensor, weight: torch.Tensor, plan: ExpertPlan, z: torch.Tensor, dys: torch.Tensor, *,
                      activation: str = "none", want=(True, True, True)):
    """(dxs, dweight, dbias) of expert_linear; `want` leaves out (None) those
    that are not needed.  z is expert_linear_forward's (None without an
    activation): float32 for float32 rows, else float16."""
    _tensors(xs=xs, weight=weight, dys=dys)
    return _native().linear_vjp(xs, weight, z, dys, activation, [bool(w) for w in want], *_arrays(plan))


def expert_combine(ys: torch.Tensor, w: torch.Tensor, plan: ExpertPlan, *,
                   residual: torch.Tensor = None) -> torch.Tensor:
    """out [tokens, width]: residual + the sum over a token's slots of
    w[token, slot] times the slot's row of ys; empty slots add nothing."""
    _tensors(ys=ys, w=w)
    return (_torch_module or _native()).combine(ys, w, residual, *_arrays(plan))


def expert_combine_vjp(ys: torch.Tensor, w: torch.Tensor, plan: ExpertPlan, dout: torch.Tensor, *,
                       want=(True, True)):
    """(dys, dw) of expert_combine; `want` leaves out (None) what is not needed."""
    _tensors(ys=ys, w=w, dout=dout)
    return _native().combine_vjp(ys, w, dout, [bool(v) for v in want], *_arrays(plan))
