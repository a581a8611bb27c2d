"""The expert operators' C ABI on the host, no device needed: every declared
function is exported, argument errors come back before anything touches a
device, and the scratch sizes."""
import os
import re

import pytest
import torch

import differentiable_exact_budget_amd as L
from differentiable_exact_budget_amd import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID = 0, 1
FAKE = 4096  # a non-NULL, 16-byte aligned address that is never dereferenced
MAX_PAIRS = 0x7FFF0000


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "lapsum_experts.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:lapsum_status_t|size_t)\s+(lapsum_\w+)\s*\(", text, re.M)
    assert sorted(names) == sorted(experts.EXPORTED)
    for name in names:
        assert hasattr(experts.lib(), name), name


def test_limits_match_the_header():
    text = open(os.path.join(ROOT, "include", "lapsum_experts.h")).read()
    value = {k: int(v, 0) for k, v in re.findall(r"#define (LAPSUM_MAX_\w+) (\w+)", text)}
    assert value == {"LAPSUM_MAX_EXPERTS": experts.MAX_EXPERTS, "LAPSUM_MAX_SLOTS": experts.MAX_SLOTS,
                     "LAPSUM_MAX_PAIRS": MAX_PAIRS}


def topk(gates=FAKE, tokens=4, E=8, m=2, floor=0.0, norm=0, ids=FAKE, w=FAKE, sums=None):
    return experts.lib().lapsum_expert_topk(gates, tokens, E, m, floor, norm, ids, w, sums, None)


@pytest.mark.parametrize("kw", [
    {"gates": None}, {"ids": None}, {"w": None}, {"tokens": -1}, {"E": 0}, {"E": 1025}, {"m": 0}, {"m": 9},
    {"E": 100, "m": 65}, {"floor": float("nan")}, {"norm": 1}, {"tokens": MAX_PAIRS // 2 + 1},
])
def test_topk_refuses(kw):
    assert topk(**kw) == INVALID


def test_calls_over_nothing():
    lib = experts.lib()
    assert topk(tokens=0, gates=None, ids=None, w=None) == OK
    assert lib.lapsum_expert_topk_vjp(None, None, None, None, 0, 8, 2, 0, None, None) == OK
    assert lib.lapsum_expert_dispatch(None, 0, 0, 2, 16, 4, None, None, None, None) == OK
    assert lib.lapsum_expert_dispatch(None, 0, 5, 2, 0, 4, None, None, None, None) == OK
    assert lib.lapsum_expert_dispatch_vjp(None, 1, 0, 2, 16, None, None, None) == OK
    assert lib.lapsum_expert_combine(None, None, None, 1, 0, 2, 16, None, None, None) == OK
    assert lib.lapsum_expert_combine_vjp(None, None, None, 1, 0, 2, 16, 4, None, None, FAKE, None, None) == OK
    assert lib.lapsum_expert_linear(None, None, None, 1, 0, 16, 16, 4, None, 0, None, None, None) == OK
    assert lib.lapsum_expert_linear(None, None, None, 1, 5, 16, 0, 4, None, 0, None, None, None) == OK


def test_vjp_of_topk_and_sort_refuse():
    lib = experts.lib()
    f = lib.lapsum_expert_topk_vjp
    assert f(None, FAKE, FAKE, FAKE, 4, 8, 2, 0, FAKE, None) == INVALID
    assert f(FAKE, FAKE, None, FAKE, 4, 8, 2, 0, FAKE, None) == INVALID
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 2, 0, None, None) == INVALID
    assert f(FAKE, None, FAKE, FAKE, 4, 8, 2, 1, FAKE, None) == INVALID
    assert f(FAKE, FAKE, FAKE, None, 4, 8, 2, 1, FAKE, None) == INVALID
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 8, 9, 1, FAKE, None) == INVALID
    s = lib.lapsum_expert_sort
    assert s(FAKE, -1, 8, FAKE, FAKE, FAKE, None, None) == INVALID
    assert s(FAKE, MAX_PAIRS + 1, 8, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert s(FAKE, 10, 0, FAKE, FAKE, FAKE, None, None) == INVALID
    assert s(FAKE, 10, 1025, FAKE, FAKE, FAKE, None, None) == INVALID
    assert s(None, 10, 8, FAKE, FAKE, FAKE, None, None) == INVALID
    assert s(FAKE, 10, 8, None, FAKE, FAKE, None, None) == INVALID
    assert s(FAKE, 10, 8, FAKE, None, FAKE, None, None) == INVALID
    assert s(FAKE, 10, 8, FAKE, FAKE, None, None, None) == INVALID
    # many workgroups need their scratch, 16-byte aligned
    assert s(FAKE, 1 << 20, 8, FAKE, FAKE, FAKE, None, None) == INVALID
    assert s(FAKE, 1 << 20, 8, FAKE, FAKE, FAKE, FAKE + 4, None) == INVALID


def test_dispatch_and_combine_refuse():
    lib = experts.lib()
    good = [FAKE, 1, 4, 2, 16, 8, FAKE, FAKE, FAKE, None]
    for at, value in ((0, None), (1, 3), (1, -1), (2, -1), (3, 0), (3, 65), (4, -1), (5, 0), (5, 1025), (6, None),
                      (7, None), (8, None), (2, MAX_PAIRS)):
        args = list(good)
        args[at] = value
        assert lib.lapsum_expert_dispatch(*args) == INVALID, (at, value)
    good = [FAKE, 1, 4, 2, 16, FAKE, FAKE, None]
    for at, value in ((0, None), (1, 3), (2, -1), (3, 65), (4, -1), (5, None), (6, None)):
        args = list(good)
        args[at] = value
        assert lib.lapsum_expert_dispatch_vjp(*args) == INVALID, (at, value)
    good = [FAKE, FAKE, None, 1, 4, 2, 16, FAKE, FAKE, None]
    for at, value in ((0, None), (1, None), (3, 9), (4, -1), (5, 0), (6, -1), (7, None), (8, None)):
        args = list(good)
        args[at] = value
        assert lib.lapsum_expert_combine(*args) == INVALID, (at, value)
    good = [FAKE, FAKE, FAKE, 1, 4, 2, 16, 8, FAKE, FAKE, FAKE, FAKE, None]
    for at, value in ((0, None), (1, None), (2, None), (3, 9), (4, -1), (5, 0), (6, -1), (7, 0), (8, None), (9, None)):
        args = list(good)
        args[at] = value
        assert lib.lapsum_expert_combine_vjp(*args) == INVALID, (at, value)
    args = list(good)
    args[10] = args[11] = None  # no output
    assert lib.lapsum_expert_combine_vjp(*args) == INVALID


def test_linear_refuses():
    lib = experts.lib()
    good = [FAKE, FAKE, None, 1, 4, 16, 16, 8, FAKE, 2, FAKE, None, None]
    for at, value in ((0, None), (1, None), (3, 3), (4, -1), (4, MAX_PAIRS + 1), (5, -1), (6, -1), (6, 1 << 31), (7, 0),
                      (7, 1025), (8, None), (9, 4), (9, -1), (10, None)):
        args = list(good)
        args[at] = value
        assert lib.lapsum_expert_linear(*args) == INVALID, (at, value)
    good = [FAKE, FAKE, FAKE, FAKE, 1, 4, 16, 16, 8, FAKE, 2, FAKE, FAKE, FAKE, FAKE, None]
    for at, value in ((0, None), (1, None), (2, None), (3, None), (4, 3), (5, -1), (6, -1), (7, -1), (8, 0), (9, None),
                      (10, 4), (14, None), (14, FAKE + 8)):
        args = list(good)
        args[at] = value
        assert lib.lapsum_expert_linear_vjp(*args) == INVALID, (at, value)
    args = list(good)
    args[11] = args[12] = args[13] = None  # no output
    assert lib.lapsum_expert_linear_vjp(*args) == INVALID


def test_scratch_sizes():
    lib = experts.lib()
    assert lib.lapsum_expert_sort_scratch_bytes(64, 8) == 0
    small, large = (lib.lapsum_expert_sort_scratch_bytes(n, 64) for n in (1 << 20, 1 << 24))
    assert 0 < small <= large <= 4 * 64 * 1025 + 256
    for bad in ((-1, 8), (MAX_PAIRS + 1, 8), (10, 0), (10, 1025)):
        assert lib.lapsum_expert_sort_scratch_bytes(*bad) == 0
    f = lib.lapsum_expert_linear_vjp_scratch_bytes
    assert f(1, 100, 16, 32, 4, 0, 0) == 0                        # dz is dys
    assert f(1, 100, 16, 32, 4, 2, 0) >= 100 * 32 * 2             # dz
    assert f(0, 100, 16, 32, 4, 2, 1) > f(0, 100, 16, 32, 4, 2, 0) >= 100 * 32 * 4
    assert f(3, 100, 16, 32, 4, 2, 1) == 0 and f(1, -1, 16, 32, 4, 2, 1) == 0


def test_tensors_on_the_host_are_refused():
    p = torch.rand(4, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    plan = L.ExpertPlan(3, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    for f in (lambda: L.expert_topk(p, 2), lambda: L.expert_sort(ids, 3), lambda: L.expert_dispatch(p, plan),
              lambda: L.expert_linear(p, torch.rand(3, 4, 8), plan),
              lambda: L.expert_combine(torch.rand(8, 4), torch.rand(4, 2), plan)):
        with pytest.raises(ValueError, match="GPU"):
            f()
