"""The C ABI of the norm, the loss and the experts' products in 8 bits on the
host, no device needed: exported functions, argument errors, scratch sizes, and
what the Python entry points refuse."""
import os
import re

import pytest
import torch

import differentiable_exact_budget_amd as L
from differentiable_exact_budget_amd import experts8, layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID = 0, 1
FAKE = 4096  # a non-NULL, 16-byte aligned address that is never dereferenced
F32, BF16, F16 = 0, 1, 2
MAX_ROWS = 0x7FFF0000


@pytest.mark.parametrize("header,module", [("lapsum_layers.h", layers), ("lapsum_experts8.h", experts8)])
def test_library_exports_every_declared_function(header, module):
    text = open(os.path.join(ROOT, "include", header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:lapsum_status_t|size_t)\s+(lapsum_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(module.EXPORTED)
    for name in names:
        assert hasattr(module.lib(), name), name


def test_limits_match_the_headers():
    text = "".join(open(os.path.join(ROOT, "include", h)).read() for h in ("lapsum_layers.h", "lapsum_experts8.h"))
    value = {k: int(v, 0) for k, v in re.findall(r"#define (LAPSUM_\w+) (\w+)", text)}
    assert value["LAPSUM_MAX_LOSS_SIDE"] == layers.MAX_LOSS_SIDE
    assert value["LAPSUM_BLOCK8"] == experts8.BLOCK
    assert value["LAPSUM_MAX_WIDTH8"] == experts8.MAX_WIDTH


def refuses(f, good, bad):
    for at, value in bad:
        args = list(good)
        args[at] = value
        assert f(*args) == INVALID, (at, value)


def test_layer_norm_refuses():
    f = layers.lib().lapsum_layer_norm
    good = [FAKE, FAKE, FAKE, BF16, F32, 4, 16, 1e-5, FAKE, FAKE, FAKE, None]
    refuses(f, good, ((0, None), (3, 3), (3, -1), (4, F16), (4, 5), (5, -1), (5, MAX_ROWS + 1), (6, 0), (6, -1),
                      (6, 1 << 31), (7, -1e-5), (7, float("nan")), (8, None)))
    assert f(None, None, None, F32, F32, 0, 16, 0.0, None, None, None, None) == OK
    f = layers.lib().lapsum_layer_norm_vjp
    good = [FAKE, FAKE, FAKE, FAKE, FAKE, F16, F32, 4, 16, FAKE, FAKE, FAKE, FAKE, None]
    refuses(f, good, ((0, None), (2, None), (3, None), (4, None), (5, 3), (6, BF16), (7, -1), (8, 0), (12, None),
                      (12, FAKE + 8)))
    args = list(good)
    args[9] = args[10] = args[11] = None  # no output
    assert f(*args) == INVALID
    args = [None] * 5 + [F32, F32, 0, 16, FAKE, None, None, None, None]
    assert f(*args) == OK


def test_linear_cross_entropy_refuses():
    side = layers.MAX_LOSS_SIDE
    f = layers.lib().lapsum_linear_cross_entropy
    good = [FAKE, FAKE, None, FAKE, BF16, 4, 100, 16, 2, FAKE, FAKE, FAKE, None]
    refuses(f, good, ((0, None), (1, None), (3, None), (4, 3), (5, -1), (5, side + 1), (6, 0), (6, -1), (6, side + 1),
                      (7, -1), (7, side + 1), (8, 3), (8, -1), (9, None), (11, None), (11, FAKE + 4)))
    assert f(None, None, None, None, F32, 0, 10, 16, 0, None, None, None, None) == OK
    f = layers.lib().lapsum_linear_cross_entropy_vjp
    good = [FAKE, FAKE, None, FAKE, FAKE, FAKE, F16, 4, 100, 16, 1, FAKE, FAKE, FAKE, FAKE, None]
    refuses(f, good, ((0, None), (1, None), (3, None), (4, None), (5, None), (6, 3), (7, -1), (7, side + 1), (8, 0),
                      (8, side + 1), (9, -1), (9, side + 1), (10, 3), (14, None), (14, FAKE + 8)))
    args = list(good)
    args[11] = args[12] = args[13] = None  # no output
    assert f(*args) == INVALID


def test_scratch_sizes():
    lib = layers.lib()
    f = lib.lapsum_layer_norm_vjp_scratch_bytes
    # partial rows of both sums, fewer than there are rows
    assert 2 * 4 * 64 <= f(BF16, 1000, 64) <= 2 * 4 * 64 * 1000
    assert f(F32, 0, 64) >= 2 * 4 * 64
    assert f(3, 10, 64) == 0 and f(F32, -1, 64) == 0 and f(F32, 10, 0) == 0
    f, b = lib.lapsum_linear_cross_entropy_scratch_bytes, lib.lapsum_linear_cross_entropy_vjp_scratch_bytes
    for bad in ((3, 10, 10, 8), (BF16, -1, 10, 8), (BF16, 10, 0, 8), (BF16, 10, 10, -1),
                (BF16, layers.MAX_LOSS_SIDE + 1, 10, 8)):
        assert f(*bad) == 0 and b(*bad) == 0
    # the logits of a large batch over a large vocabulary are not kept
    for dtype in (F32, BF16, F16):
        assert f(dtype, 8192, 262144, 2048) < 8192 * 262144 * 2 / 8
        assert b(dtype, 8192, 262144, 2048) < 8192 * 262144 * 2 / 4


def test_rows_in_8_bits_refuse():
    lib = experts8.lib()
    good = [FAKE, BF16, 4, 200, FAKE, FAKE, None]
    refuses(lib.lapsum_expert_quantize, good, ((0, None), (1, 3), (2, -1), (2, MAX_ROWS + 1), (3, -1), (3, MAX_ROWS + 1),
                                               (4, None), (4, FAKE + 8), (5, None)))
    good = [FAKE, FAKE, BF16, 4, 200, FAKE, None]
    refuses(lib.lapsum_expert_dequantize, good, ((0, None), (0, FAKE + 4), (1, None), (2, 3), (3, -1), (4, -1), (5, None)))
    assert lib.lapsum_expert_quantize(None, F32, 0, 200, None, None, None) == OK
    assert lib.lapsum_expert_dequantize(None, None, F32, 7, 0, None, None) == OK
    good = [FAKE, FAKE, FAKE, FAKE, None, BF16, 4, 256, 64, 8, FAKE, 2, FAKE, None]
    refuses(lib.lapsum_expert_linear_fp8, good,
            ((0, None), (0, FAKE + 8), (1, None), (2, None), (2, FAKE + 8), (3, None), (5, 3), (6, -1), (6, MAX_ROWS + 1),
             (7, -1), (7, experts8.MAX_WIDTH + 1), (8, -1), (8, MAX_ROWS + 1), (9, 0), (9, 1025), (10, None), (11, 4),
             (11, -1), (12, None)))
    # more tiles than a launch holds
    args = list(good)
    args[6], args[8] = 1 << 24, 1 << 17
    assert lib.lapsum_expert_linear_fp8(*args) == INVALID
    args[6], args[8] = 1, MAX_ROWS
    assert lib.lapsum_expert_linear_fp8(*args) == INVALID


def test_tensors_on_the_host_are_refused():
    x = torch.rand(4, 128)
    rows = L.ScaledRows(torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.ones(4, 1).to(torch.float8_e8m0fnu), 128)
    plan = L.ExpertPlan(1, torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                        torch.zeros(4, 1, dtype=torch.int32))
    for f in (lambda: L.layer_norm(x), lambda: L.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int64)),
              lambda: L.expert_quantize(x), lambda: L.expert_dequantize(rows),
              lambda: L.expert_linear_fp8(rows, rows, plan)):
        with pytest.raises(ValueError, match="GPU"):
            f()


def test_other_types_are_refused():
    x = torch.rand(4, 128)
    for f in (lambda: L.layer_norm([1.0]), lambda: L.linear_cross_entropy(x, None, x), lambda: L.expert_quantize(1.0),
              lambda: L.expert_dequantize(x), lambda: L.expert_linear_fp8(x, x, None)):
        with pytest.raises(TypeError):
            f()
