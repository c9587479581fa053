"""Autograd under stream capture (no GPU): recording a call and running its
backward pass are refused, each by itself, and without a gradient nothing is."""

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
    """Host tensors pass as device ones; what would launch is listed by name."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    for name in ("mm_sort_tokens", "mm_sort_rows", "mm_combine_tokens", "mm_combine_backward", "mm_swiglu", "mm_swiglu_backward"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append(name))
    return seen


@pytest.fixture
def capturing(monkeypatch):
    """Sets whether the current stream is being captured."""
    now = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0])
    return lambda on: now.__setitem__(0, on)


def calls():
    """name -> (a call, the inputs that require a gradient)"""
    ids = torch.randint(0, E, (T, K), dtype=torch.int32)
    order = moe.TokenOrder(*ref.order(ids, E))
    leaf = lambda *shape: torch.zeros(*shape, requires_grad=True)
    x, rows, w, h = leaf(T, H), leaf(T * K, H), leaf(T, K), leaf(3, 16)
    fixed = torch.zeros(T * K, H)
    return {
        "sort_tokens": (lambda: moe.sort_tokens(x, ids, E)[0], (x,)),
        "sort_rows": (lambda: moe.sort_rows(x, order), (x,)),
        "combine_tokens": (lambda: moe.combine_tokens(rows, order), (rows,)),
        "combine_tokens of both": (lambda: moe.combine_tokens(rows, order, w), (rows, w)),
        "combine_tokens of weights": (lambda: moe.combine_tokens(fixed, order, w), (w,)),
        "swiglu": (lambda: moe.swiglu(h), (h,)),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_recorded_under_capture(launches, capturing, name):
    call, _ = calls()[name]
    capturing(True)
    with pytest.raises(RuntimeError, match="capture"):
        call()
    assert not launches
    with torch.no_grad():
        assert call().grad_fn is None
    assert len(launches) == 1


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("create_graph", [False, True])
def test_backward_under_capture(launches, capturing, name, create_graph):
    call, inputs = calls()[name]
    capturing(False)
    y = call()
    capturing(True)
    n = len(launches)
    with pytest.raises(RuntimeError, match="capture"):
        torch.autograd.grad(y, inputs, torch.ones_like(y), retain_graph=True, create_graph=create_graph)
    assert len(launches) == n
    capturing(False)
    got = torch.autograd.grad(y, inputs, torch.ones_like(y), create_graph=create_graph)
    assert [g.shape for g in got] == [t.shape for t in inputs] and len(launches) == n + 1
