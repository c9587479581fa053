"""Host side of the token sort (no GPU): plans, their limits, refusals before
any HIP call, and how the functions read their arguments."""

from __future__ import annotations

import contextlib
import ctypes
import os

import pytest
import torch

import sort_reference as ref
from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

GOOD = 1 << 20          # an aligned fake address; never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.lib_path()):
        from mixture_experts_expert_mm_amd import _build
        _build.build()
    return B.load()


def test_plan():
    assert ctypes.sizeof(B.MMSortProblem) == 40 and ctypes.sizeof(B.MMSortPlan) == 40 + 8 + 8 + 32
    assert B.mm_sort_plan_create(1, 1, 1, 1, 0).workspace_bytes == 0
    assert B.mm_sort_plan_create(16384, 7168, 256, 8, 0).workspace_bytes >= 128 * 256 * 4
    assert B.mm_sort_plan_create(1 << 24, 8, 1024, 63, 3).workspace_bytes >= 512 * 1024 * 4


@pytest.mark.parametrize("dims", [(0, 8, 4, 2), ((1 << 24) + 1, 8, 4, 2), (4, 0, 4, 2), (4, (1 << 20) + 1, 4, 2), (4, 8, 0, 2),
                                  (4, 8, 1025, 2), (4, 8, 4, 0), (4, 8, 4, 65), (1 << 24, 8, 4, 64)])
def test_plan_refuses(dims):
    with pytest.raises(B.MMError) as ei:
        B.mm_sort_plan_create(*dims, 0)
    assert ei.value.status == 1


def test_entry_points_validate_before_any_hip_call(lib):
    P = ctypes.byref
    for element in (-1, 4):
        with pytest.raises(B.MMError) as ei:
            B.mm_sort_plan_create(4, 8, 4, 2, element)
        assert ei.value.status == 2

    def call(fn, args, i, v):
        a = list(args)
        a[i] = v
        return fn(*a)

    sp = B.mm_sort_plan_create(5000, 8, 4, 2, 0)
    bad = B.MMSortPlan.from_buffer_copy(sp)
    bad.prob.num_topk = 1
    args = [P(sp), GOOD, None, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 1 << 40, None]
    for i in (1, 4, 5, 6, 7, 9):
        assert call(lib.mm_sort_tokens, args, i, None) == 1
        assert call(lib.mm_sort_tokens, args, i, GOOD + 2) == 1
    assert call(lib.mm_sort_tokens, args, 3, None) == 1            # x and rows: both or neither
    assert call(lib.mm_sort_tokens, args, 8, None) == 1
    assert call(lib.mm_sort_tokens, args, 8, GOOD + 4) == 1
    assert call(lib.mm_sort_tokens, args, 10, 16) == 3
    for p in (P(bad), None):
        assert call(lib.mm_sort_tokens, args, 0, p) == 1
    args = [P(sp), GOOD, GOOD, GOOD, GOOD, None]
    for i in (1, 2, 3, 4):
        assert call(lib.mm_sort_rows, args, i, None) == 1
        assert call(lib.mm_sort_rows, args, i, GOOD + 2) == 1
    args = [P(sp), GOOD, GOOD, GOOD, GOOD, None]
    for i in (1, 2, 4):
        assert call(lib.mm_combine_tokens, args, i, None) == 1
        assert call(lib.mm_combine_tokens, args, i, GOOD + 2) == 1
    assert call(lib.mm_combine_tokens, args, 3, GOOD + 2) == 1
    codes = B.mm_sort_plan_create(5000, 8, 4, 2, B.MM_ELEMENT_8BIT)
    assert call(lib.mm_combine_tokens, args, 0, P(codes)) == 2     # codes have no sums
    args = [P(sp), GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None]
    for i in (1, 2, 3, 4, 5):
        assert call(lib.mm_combine_backward, args, i, None) == 1
        assert call(lib.mm_combine_backward, args, i, GOOD + 2) == 1
    assert call(lib.mm_combine_backward, args, 6, GOOD + 4) == 1
    assert call(lib.mm_combine_backward, args, 7, GOOD + 2) == 1
    assert call(lib.mm_combine_backward, args, 0, P(codes)) == 2
    args[6] = args[7] = None
    assert lib.mm_combine_backward(*args) == 1                     # nothing to compute
    assert [B.mm_kernel_name(i) for i in range(17, 21)] == ["sort_order", "sort_rows", "combine_tokens", "combine_backward"]


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; the calls that would launch are listed as (name, arguments)."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    for name in ("mm_sort_tokens", "mm_sort_rows", "mm_combine_tokens", "mm_combine_backward"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def some(T=6, E=4, K=2, H=8):
    ids = torch.randint(0, E, (T, K), dtype=torch.int32)
    return ids, moe.TokenOrder(*ref.order(ids, E)), torch.zeros(T, H), torch.zeros(T * K, H), torch.rand(T, K)


def test_what_is_launched(launches):
    ids, order, x, rows, w = some()
    r, o = moe.sort_tokens(x, ids, 4)
    assert r.shape == rows.shape and r.dtype == x.dtype and o.offsets.shape == (5,)
    assert launches[-1][0] == "mm_sort_tokens" and launches[-1][1][9] is None          # few routes: no workspace
    big = torch.zeros(5000, 2, dtype=torch.int32)
    moe.sort_tokens(torch.zeros(5000, 8, dtype=torch.int8), big, 4)
    assert launches[-1][1][9].numel() == launches[-1][1][0].workspace_bytes
    moe.sort_rows(x, order)
    moe.combine_tokens(rows, order)
    assert launches[-1][1][3] is None
    d, dw = moe.combine_backward(x, rows, order, w)
    assert d.shape == rows.shape and dw.dtype == torch.float32 and dw.shape == w.shape
    assert [n for n, _ in launches[2:]] == ["mm_sort_rows", "mm_combine_tokens", "mm_combine_backward"]


def test_refusals(launches):
    ids, order, x, rows, w = some()
    bad = [
        ("x", lambda: moe.sort_tokens(x.double(), ids, 4)), ("x", lambda: moe.sort_tokens(x[:, ::2], ids, 4)),
        ("topk_ids", lambda: moe.sort_tokens(x, ids.long(), 4)), ("topk_ids", lambda: moe.sort_tokens(x, ids[:5], 4)),
        ("topk_ids", lambda: moe.sort_tokens(x, ids.t(), 4)), ("topk_ids", lambda: moe.sort_tokens(x, None, 4)),
        ("active", lambda: moe.sort_tokens(x, ids, 4, active=torch.ones(6))),
        ("num_experts", lambda: moe.sort_tokens(x, ids, 4.5)), ("order", lambda: moe.sort_rows(x, None)),
        ("order", lambda: moe.sort_rows(x[:5], order)), ("rows", lambda: moe.combine_tokens(rows[:5], order)),
        ("rows", lambda: moe.combine_tokens(rows.to(torch.int8), order)),
        ("weights", lambda: moe.combine_tokens(rows, order, w.to(torch.bfloat16))),
        ("weights", lambda: moe.combine_tokens(rows, order, w[:, :1])),
        ("weights", lambda: moe.combine_backward(x, rows, order, None)),
        ("dy", lambda: moe.combine_backward(x.half(), rows, order, w)), ("dy", lambda: moe.combine_backward(x[:2], rows, order, w)),
        ("order.offsets", lambda: moe.sort_rows(x, moe.TokenOrder(order.counts, None, order.row_of_route, order.route_of_row))),
        ("order.offsets", lambda: moe.sort_rows(x, moe.TokenOrder(order.counts, order.offsets.long(), order.row_of_route, order.route_of_row))),
        ("order.row_of_route", lambda: moe.sort_rows(x, moe.TokenOrder(order.counts, order.offsets, order.row_of_route.view(-1), order.route_of_row))),
        ("order.row_of_route", lambda: moe.combine_tokens(rows, moe.TokenOrder(order.counts, order.offsets, order.row_of_route.float(), order.route_of_row))),
        ("order.row_of_route", lambda: moe.combine_tokens(rows, moe.TokenOrder(order.counts, order.offsets, order.row_of_route.t(), order.route_of_row))),
        ("rows: .*gradient", lambda: moe.combine_backward(x, rows.clone().requires_grad_(), order, w)),
        ("weights: .*gradient", lambda: moe.combine_backward(x, rows, order, w.clone().requires_grad_())),
    ]
    for match, call in bad:
        with pytest.raises(ValueError, match="^" + match):
            call()
    for E in (0, 1025):
        with pytest.raises(B.MMError):
            moe.sort_tokens(x, ids, E)
    with pytest.raises(B.MMError):
        moe.sort_tokens(x[:, :0], ids, 4)
    assert not launches
    import torch.autograd.forward_ad as fw
    with fw.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            moe.sort_tokens(fw.make_dual(x, x), ids, 4)


def test_host_tensors_are_refused():
    ids, order, x, rows, w = some()
    for call in (lambda: moe.sort_tokens(x, ids, 4), lambda: moe.sort_rows(x, order), lambda: moe.combine_tokens(rows, order),
                 lambda: moe.combine_backward(x, rows, order, w)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
