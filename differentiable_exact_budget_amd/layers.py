"""The norm in front of a routed layer and the loss behind it.

    h = layer_norm(x, weight, bias)                        # rows of a router and its experts
    loss = linear_cross_entropy(h, vocabulary, target)     # softmax cross entropy of h @ vocabulary.T

Both are differentiable, once and in reverse mode (second derivatives and
forward-mode tangents are refused, and so is torch.jit.trace); each gradient
also has an entry point of its own (*_vjp).  They run in liblapsum.so
(hand-written HIP for gfx950, the C ABI of include/lapsum_layers.h) on the
caller's current stream, never wait for the device and can be captured into a
graph (of a backward pass, while no eager graph of the same leaves is alive:
autograd would wait for those leaves' stream inside the capture).

Rows may be float32, bfloat16 or float16.  Statistics and sums are held in
float32 and rounded once to the rows' type.
"""
import ctypes

import torch

from . import _binding
from .experts import _native, _tensors

__all__ = ["layer_norm", "layer_norm_forward", "layer_norm_vjp", "linear_cross_entropy",
           "linear_cross_entropy_forward", "linear_cross_entropy_vjp", "MAX_LOSS_SIDE"]

MAX_LOSS_SIDE = 0x1000000

EXPORTED = [
    "lapsum_layer_norm", "lapsum_layer_norm_vjp_scratch_bytes", "lapsum_layer_norm_vjp",
    "lapsum_linear_cross_entropy_scratch_bytes", "lapsum_linear_cross_entropy",
    "lapsum_linear_cross_entropy_vjp_scratch_bytes", "lapsum_linear_cross_entropy_vjp",
]

_lib = None


def lib():
    """ctypes view of the operators' C ABI in liblapsum.so."""
    global _lib
    if _lib is None:
        L = _binding.lib()
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        types = {
            "lapsum_layer_norm": [vp, vp, vp, i32, i32, i64, i64, f32, vp, vp, vp, vp],
            "lapsum_layer_norm_vjp_scratch_bytes": [i32, i64, i64],
            "lapsum_layer_norm_vjp": [vp, vp, vp, vp, vp, i32, i32, i64, i64, vp, vp, vp, vp, vp],
            "lapsum_linear_cross_entropy_scratch_bytes": [i32, i64, i64, i64],
            "lapsum_linear_cross_entropy": [vp, vp, vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, vp],
            "lapsum_linear_cross_entropy_vjp_scratch_bytes": [i32, i64, i64, i64],
            "lapsum_linear_cross_entropy_vjp": [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp],
        }
        for name, args in types.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_size_t if name.endswith("_bytes") else ctypes.c_int
        _lib = L
    return _lib


def layer_norm(x: torch.Tensor, weight: torch.Tensor = None, bias: torch.Tensor = None, *,
               eps: float = 1e-5) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension of
    x, which has at least one element.

    weight and bias have x's last dimension and either x's dtype or float32
    (both the same); None stands for 1 and 0.  Statistics are float32, the
    variance from values about the mean; one past float32's range is infinite,
    and the row's result the bias."""
    _tensors(x=x)
    return _native().layer_norm(x, weight, bias, eps)


def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor = None, bias: torch.Tensor = None, *, eps: float = 1e-5):
    """(y, mean, rstd) of layer_norm, outside autograd: the mean and 1 /
    sqrt(var + eps) of every row, float32, are what layer_norm_vjp wants."""
    _tensors(x=x)
    return _native().layer_norm_forward(x, weight, bias, eps)


def layer_norm_vjp(x: torch.Tensor, weight, mean: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor, *,
                   want=(True, True, True)):
    """(dx, dweight, dbias) of layer_norm; `want` leaves out (None) those that
    are not needed.  dweight and dbias have weight's dtype (x's where weight is
    None) and are summed over the rows in float32."""
    _tensors(x=x, mean=mean, rstd=rstd, dy=dy)
    return _native().layer_norm_vjp(x, weight, mean, rstd, dy, [bool(w) for w in want])


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, *, bias: torch.Tensor = None,
                         reduction: str = "mean") -> torch.Tensor:
    """Softmax cross entropy of the logits x @ weight.T + bias, which are never
    kept: log(sum(exp(z))) - z[target], float32.

    x [..., width], weight [vocabulary, width] and bias [vocabulary] or None
    have one dtype; target [...] is int64.  A row whose target is outside [0,
    vocabulary) is ignored: its loss is 0, it has no gradient, and the mean does
    not count it (and is 0 where no row counts), whatever it holds.  reduction is "none", "sum" or
    "mean".  A bias of -inf takes an entry out of the vocabulary; a row with a
    logit of +inf or NaN, or with nothing but -inf, has a loss of NaN or inf.

    Differentiable with respect to x, weight and bias.  The logits are formed
    again for the gradient, a piece of the vocabulary at a time; their gradient,
    over the largest gradient of a row's loss, is rounded once to the rows' type
    for the products that follow (x's and weight's gradients), which hold their
    sums and that factor in float32; bias' is summed before that rounding."""
    _tensors(x=x, weight=weight, target=target)
    return _native().linear_cross_entropy(x, weight, target, bias, reduction)


def linear_cross_entropy_forward(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, *,
                                 bias: torch.Tensor = None, reduction: str = "mean"):
    """(loss, lse) of linear_cross_entropy, outside autograd: lse, float32 and
    shaped as target, is the logarithm that linear_cross_entropy_vjp wants."""
    _tensors(x=x, weight=weight, target=target)
    return _native().linear_cross_entropy_forward(x, weight, target, bias, reduction)


def linear_cross_entropy_vjp(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                             dloss: torch.Tensor, *, bias: torch.Tensor = None, reduction: str = "mean",
                             want=(True, True, False)):
    """(dx, dweight, dbias) of linear_cross_entropy from dloss, float32 and
    shaped as the loss; `want` leaves out (None) those that are not needed."""
    _tensors(x=x, weight=weight, target=target, lse=lse, dloss=dloss)
    return _native().linear_cross_entropy_vjp(x, weight, target, lse, dloss, bias, reduction, [bool(w) for w in want])
