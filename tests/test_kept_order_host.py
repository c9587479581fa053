"""What the differentiable functions keep for their backward pass (no GPU): the
tensors of the forward call, whatever the program does with its objects in
between.  The launches are recorded, with the tensors that they were given."""

from __future__ import annotations

import contextlib

import pytest
import torch

import sort_reference as ref
from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

T, E, K, H = 6, 4, 2, 8


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; the calls that would launch are listed as (name, arguments)."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(moe, "_not_captured", lambda: None)
    for name in ("mm_sort_tokens", "mm_sort_rows", "mm_combine_tokens", "mm_combine_backward", "mm_swiglu", "mm_swiglu_backward"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def order(tokens=T, seed=0):
    ids = torch.randint(0, E, (tokens, K), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    return moe.TokenOrder(*ref.order(ids, E))


def recorded(o, kind):
    """(output, inputs that require a gradient, the backward launch's name, where it is given offsets and rows of routes)"""
    if kind == "sort":
        x = torch.zeros(T, H, requires_grad=True)
        return moe.sort_rows(x, o), (x,), "mm_combine_tokens", None, 2
    rows = torch.zeros(T * K, H, requires_grad=True)
    if kind == "combine":
        return moe.combine_tokens(rows, o), (rows,), "mm_sort_rows", 2, 3
    w = torch.zeros(T, K, requires_grad=True)
    return moe.combine_tokens(rows, o, w), (rows, w), "mm_combine_backward", 3, 4


KINDS = ["sort", "combine", "weighted"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [T, 3])
def test_an_order_whose_fields_are_new_tensors(launches, kind, tokens):
    """An object that the next micro-batch fills anew: the gradient goes by the order of the forward call."""
    o = order()
    offsets, row = o.offsets, o.row_of_route
    y, of, name, at, at_row = recorded(o, kind)
    other = order(tokens, seed=1)
    o.counts, o.offsets, o.row_of_route, o.route_of_row = other.counts, other.offsets, other.row_of_route, other.route_of_row
    torch.autograd.grad(y, of, torch.ones_like(y))
    got, args = launches[-1]
    assert got == name and args[0].prob.num_tokens == T
    assert args[at_row].data_ptr() == row.data_ptr() and args[at_row].shape == (T, K)
    assert at is None or args[at].data_ptr() == offsets.data_ptr()


@pytest.mark.parametrize("kind", KINDS)
def test_an_order_that_is_written_over(launches, kind):
    o = order()
    y, of, *_ = recorded(o, kind)
    o.row_of_route.zero_()
    n = len(launches)
    with pytest.raises(RuntimeError, match="modified in place"):
        torch.autograd.grad(y, of, torch.ones_like(y))
    assert len(launches) == n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("field,other", [("row_of_route", torch.zeros(3, K, dtype=torch.int32)),
                                         ("row_of_route", torch.zeros(T, K, dtype=torch.int64)),
                                         ("row_of_route", torch.zeros(K, T, dtype=torch.int32).t())])
def test_data_that_is_exchanged(launches, kind, field, other):
    """t.data = ... passes autograd's own check; what would be read out of bounds is refused."""
    o = order()
    y, of, *_ = recorded(o, kind)
    getattr(o, field).data = other
    n = len(launches)
    with pytest.raises((RuntimeError, ValueError), match=field):
        torch.autograd.grad(y, of, torch.ones_like(y))
    assert len(launches) == n


def test_rows_and_weights_that_are_exchanged(launches):
    for name in ("rows", "weights"):
        rows, w = torch.zeros(T * K, H, requires_grad=True), torch.zeros(T, K, requires_grad=True)
        y = moe.combine_tokens(rows, order(), w)
        t = rows if name == "rows" else w
        t.data = t.data[:3].clone()
        n = len(launches)
        with pytest.raises((RuntimeError, ValueError), match=name):
            torch.autograd.grad(y, (rows, w), torch.ones_like(y))
        assert len(launches) == n


@pytest.mark.parametrize("kind", KINDS)
def test_an_order_made_in_inference_mode(launches, kind):
    """Routes that were sorted ahead of the training step: their order serves it like another."""
    with torch.inference_mode():
        made = order()
        o = moe.TokenOrder(*(t.clone() for t in (made.counts, made.offsets, made.row_of_route, made.route_of_row)))
    assert o.row_of_route.is_inference()
    y, of, name, at, at_row = recorded(o, kind)
    torch.autograd.grad(y, of, torch.ones_like(y))
    got, args = launches[-1]
    assert got == name and torch.equal(args[at_row], o.row_of_route)
    assert at is None or torch.equal(args[at], o.offsets)


@pytest.mark.parametrize("kind", KINDS)
def test_hooks_of_saved_tensors_see_the_order(launches, kind):
    """A program that moves what is kept elsewhere moves the order too, and a copy comes back."""
    o, packed = order(), []

    def pack(t):
        packed.append(t)
        return t.clone()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y, of, name, at, at_row = recorded(o, kind)
    assert any(t.data_ptr() == o.row_of_route.data_ptr() for t in packed)
    torch.autograd.grad(y, of, torch.ones_like(y))
    got, args = launches[-1]
    assert got == name and torch.equal(args[at_row], o.row_of_route) and args[at_row].data_ptr() != o.row_of_route.data_ptr()


def test_hooks_that_bring_something_else_back(launches):
    """A kept copy of another type or size would be read out of bounds."""
    for back in (lambda t: t.half() if t.is_floating_point() else t, lambda t: t[:1]):
        for call in (lambda: moe.swiglu(torch.zeros(3, 16, requires_grad=True)), lambda: recorded(order(), "weighted")[0]):
            with torch.autograd.graph.saved_tensors_hooks(lambda t: t, back):
                y = call()
            n = len(launches)
            with pytest.raises((RuntimeError, ValueError), match="is needed"):
                y.sum().backward()
            assert len(launches) == n


@pytest.mark.parametrize("kind", KINDS)
def test_the_order_is_let_go(launches, kind):
    """A backward pass that keeps no graph releases what was kept for it."""
    o = order()
    y, of, *_ = recorded(o, kind)
    torch.autograd.grad(y, of, torch.ones_like(y))
    with pytest.raises(RuntimeError, match="second time|already been freed"):
        torch.autograd.grad(y, of, torch.ones_like(y))
