"""The four tensors of an order stand by themselves (no GPU): what a program
writes into one is no change of the others for autograd."""

from __future__ import annotations

import contextlib

import pytest
import torch

from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

FIELDS = ["counts", "offsets", "row_of_route", "route_of_row"]
READ = {"rows": {"offsets", "row_of_route"}, "x": {"row_of_route"}}       # by which gradient


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; the calls that would launch are listed by name."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(moe, "_not_captured", lambda: None)
    for name in ("mm_sort_tokens", "mm_sort_rows", "mm_combine_tokens", "mm_combine_backward"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append(name))
    return seen


@pytest.mark.parametrize("T", [6, 0])
@pytest.mark.parametrize("field", FIELDS)
@pytest.mark.parametrize("of", ["x", "rows"])
def test_a_field_that_is_written_over(launches, T, field, of):
    x, ids, w = torch.zeros(T, 8, requires_grad=True), torch.zeros(T, 2, dtype=torch.int32), torch.zeros(T, 2)
    rows, o = moe.sort_tokens(x, ids, 4)
    assert [tuple(getattr(o, f).shape) for f in FIELDS] == [(4,), (5,), (T, 2), (2 * T,)]
    assert all(getattr(o, f).is_contiguous() for f in FIELDS)
    leaf = torch.zeros(2 * T, 8, requires_grad=True)
    y, inputs = (rows, x) if of == "x" else (moe.combine_tokens(leaf, o, w), leaf)
    getattr(o, field).add_(1)
    if field in READ[of]:
        with pytest.raises(RuntimeError, match=field):
            torch.autograd.grad(y, inputs, torch.ones_like(y))
    else:
        assert torch.autograd.grad(y, inputs, torch.ones_like(y))[0].shape == inputs.shape


@pytest.mark.parametrize("T", [6, 0])
def test_one_field_is_not_another_ones_memory(launches, T):
    ids = torch.zeros(T, 2, dtype=torch.int32)
    _, o = moe.sort_tokens(torch.zeros(T, 8), ids, 4)
    for i, f in enumerate(FIELDS):
        getattr(o, f).fill_(i + 1)
    assert all(bool((getattr(o, f) == i + 1).all()) for i, f in enumerate(FIELDS))
