"""The experts' products in 8 bits, for serving.

    weight = expert_quantize(w)                            # once: [experts, out, in]
    xs = expert_quantize(expert_dispatch(x, plan))
    ys = expert_linear_fp8(xs, weight, plan, activation="silu")

Rows in 8 bits are e4m3 values in blocks of 128 along the row, each block under
a power of two: half the bytes of 16-bit rows and twice the matrix rate.  These
operators have no gradients.  They run in liblapsum.so (hand-written HIP for
gfx950, the C ABI of include/lapsum_experts8.h) on the caller's current stream,
never wait for the device and can be captured into a graph.
"""
import ctypes

import torch

from . import _binding
from .experts import _arrays, _native, _tensors

__all__ = ["ScaledRows", "expert_quantize", "expert_dequantize", "expert_linear_fp8", "BLOCK", "MAX_WIDTH"]

BLOCK = 128
MAX_WIDTH = 0x100000

EXPORTED = ["lapsum_expert_quantize", "lapsum_expert_dequantize", "lapsum_expert_linear_fp8"]

_lib = None


def lib():
    """ctypes view of the operators' C ABI in liblapsum.so."""
    global _lib
    if _lib is None:
        L = _binding.lib()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        types = {
            "lapsum_expert_quantize": [vp, i32, i64, i64, vp, vp, vp],
            "lapsum_expert_dequantize": [vp, vp, i32, i64, i64, vp, vp],
            "lapsum_expert_linear_fp8": [vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, vp, i32, vp, vp],
        }
        for name, args in types.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _lib = L
    return _lib


class ScaledRows:
    """Rows in 8 bits, as expert_quantize makes them.

    values [..., blocks * 128], float8_e4m3fn, zeros past `width`; scales [...,
    blocks], float8_e8m0fnu (powers of two); blocks = ceil(width / 128).  Both
    are contiguous and values start on 16 bytes.  An element stands for its
    value times its block's scale."""
    __slots__ = ("values", "scales", "width")

    def __init__(self, values: torch.Tensor, scales: torch.Tensor, width: int):
        self.values, self.scales, self.width = values, scales, width

    @property
    def shape(self):
        return self.values.shape[:-1] + (self.width,)


def _rows(name, rows):
    if not isinstance(rows, ScaledRows):
        raise TypeError(f"{name} must be ScaledRows")
    _tensors(**{f"{name}.values": rows.values, f"{name}.scales": rows.scales})
    return rows.values, rows.scales, rows.width


def expert_quantize(x: torch.Tensor) -> ScaledRows:
    """x [..., width] (float32, bfloat16 or float16) in 8 bits.  A block's
    scale is the least power of two 2^e (e >= -127; 1 for a block of zeros) with which
    its largest finite magnitude is at most 448, and a value is x / 2^e to the
    nearest e4m3, ties to even.  Infinities and NaN become NaN and do not count
    for the scale."""
    _tensors(x=x)
    return ScaledRows(*_native().quantize(x), x.shape[-1])


def expert_dequantize(rows: ScaledRows, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """What rows in 8 bits stand for, rounded to dtype: float32, bfloat16 or
    float16 (where a value past 65504 is infinite)."""
    return _native().dequantize(*_rows("rows", rows), dtype)


def expert_linear_fp8(xs: ScaledRows, weight: ScaledRows, plan, *, bias: torch.Tensor = None,
                      activation: str = "none", dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """ys [rows, out] of dtype: act(xs W_e^T + b_e), e the expert of each row
    by the plan; zeros past the used rows.  xs [rows, in] and weight [experts,
    out, in] are rows in 8 bits, bias [experts, out] is of dtype or None.

    float32 results have exact products and float32 sums.  16-bit results come
    from the 8-bit matrix instruction, which drops, of eight neighbouring
    products along the sum, what is below 2^-13 of the largest one's power of two
    (random rows: 1.5e-5 of the result in the 2-norm), and sums those in float32.

    No gradient: a bias that requires one is refused."""
    return _native().linear_fp8(*_rows("xs", xs), *_rows("weight", weight), bias, activation, dtype, *_arrays(plan))
