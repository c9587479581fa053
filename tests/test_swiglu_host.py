"""Host side of the activation (no GPU): refusals before any HIP call and how
its functions read their arguments."""

from __future__ import annotations

import contextlib
import os

import pytest
import torch

from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

GOOD = 1 << 20          # an aligned fake address; never dereferenced on these paths


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.lib_path()):
        from mixture_experts_expert_mm_amd import _build
        _build.build()
    return B.load()


def test_entry_points_validate_before_any_hip_call(lib):
    fwd = [4, 8, 0, 0, GOOD, 0, 0.0, GOOD, GOOD, GOOD, None]
    bwd = [4, 8, 0, 0, GOOD, GOOD, GOOD, 0, 0.0, GOOD, None]

    def call(fn, args, *changes):
        a = list(args)
        for i, v in changes:
            a[i] = v
        return fn(*a)

    for fn, args in ((lib.mm_swiglu, fwd), (lib.mm_swiglu_backward, bwd)):
        for i, v in ((0, 0), (0, (1 << 24) + 1), (1, 0), (1, (1 << 20) + 1)):
            assert call(fn, args, (i, v)) == 1
        assert call(fn, args, (0, 1 << 24), (1, 1 << 14)) == 1                 # 2^31 groups
        for v in (-1, 3, 4):
            assert call(fn, args, (2, v)) == 2
        for cols, v in ((8, -8), (8, 4), (8, 16), (40, 32), (24, 12)):             # groups of gate and up columns
            assert call(fn, args, (1, cols), (3, v)) == 1
    for on, c in ((2, 0.0), (1, -1.0), (1, float("nan"))):
        assert call(lib.mm_swiglu, fwd, (5, on), (6, c)) == 1
        assert call(lib.mm_swiglu_backward, bwd, (7, on), (8, c)) == 1
    for i in (4, 7):
        assert call(lib.mm_swiglu, fwd, (i, None)) == 1 and call(lib.mm_swiglu, fwd, (i, GOOD + 8)) == 1
    for i, v in ((8, None), (9, None), (8, GOOD + 8), (9, GOOD + 2)):          # codes and scales: both or neither
        assert call(lib.mm_swiglu, fwd, (i, v)) == 1
    for i in (4, 5, 6, 9):
        assert call(lib.mm_swiglu_backward, bwd, (i, None)) == 1
        assert call(lib.mm_swiglu_backward, bwd, (i, GOOD + 2)) == 1
    assert [B.mm_kernel_name(i) for i in (21, 22)] == ["swiglu", "swiglu_backward"]


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; the calls that would launch are listed as (name, arguments)."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(moe, "_not_captured", lambda: None)
    for name in ("mm_swiglu", "mm_swiglu_backward"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def test_what_is_launched(launches):
    h = torch.zeros(3, 520, dtype=torch.bfloat16)
    assert moe.swiglu(h).shape == (3, 260) and launches[-1][1][7] is None      # nothing is kept
    a, q, s = moe.swiglu_forward(h, activation_clamp=2)
    assert q.shape == h.shape and q.dtype == torch.int8 and s.shape == (3, 6) and launches[-1][1][5] == 2.0
    moe.swiglu(h.clone().requires_grad_())
    assert launches[-1][1][7] is not None
    with torch.no_grad():
        moe.swiglu(h.clone().requires_grad_())
    assert launches[-1][1][7] is None
    assert moe.swiglu_backward(a, q, s).shape == h.shape
    n = len(launches)
    assert moe.swiglu(h[:0]).shape == (0, 260) and len(launches) == n


def test_refusals(launches):
    h = torch.zeros(3, 520, dtype=torch.bfloat16)
    q, s, da = torch.zeros(3, 520, dtype=torch.int8), torch.zeros(3, 6), torch.zeros(3, 260, dtype=torch.bfloat16)
    bad = [
        ("h", lambda: moe.swiglu(h.double())), ("h", lambda: moe.swiglu(q)), ("h", lambda: moe.swiglu(h[:, ::2])),
        ("h", lambda: moe.swiglu(h[:, :5].contiguous())), ("h", lambda: moe.swiglu(h[:, :0])),
        ("h: .*gradient", lambda: moe.swiglu_forward(h.clone().requires_grad_())),
        ("activation_clamp", lambda: moe.swiglu(h, activation_clamp=-1.0)),
        ("activation_clamp", lambda: moe.swiglu(h, activation_clamp=float("nan"))),
        ("activation_clamp", lambda: moe.swiglu_backward(da, q, s, activation_clamp=-2)),
        ("gate_up_group", lambda: moe.swiglu(h, gate_up_group=12)), ("gate_up_group", lambda: moe.swiglu(h, gate_up_group=32)),
        ("gate_up_group", lambda: moe.swiglu(h, gate_up_group=-8)), ("gate_up_group", lambda: moe.swiglu(h, gate_up_group=1.5)),
        ("gate_up_group", lambda: moe.swiglu_backward(da, q, s, gate_up_group=8)),
        ("da", lambda: moe.swiglu_backward(da.double(), q, s)), ("codes", lambda: moe.swiglu_backward(da, q[:2], s)),
        ("codes", lambda: moe.swiglu_backward(da, h, s)), ("scales", lambda: moe.swiglu_backward(da, q, s[:, :5])),
        ("scales", lambda: moe.swiglu_backward(da, q, s.half())), ("da", lambda: moe.swiglu_backward(da.t(), q, s)),
        ("scales: .*gradient", lambda: moe.swiglu_backward(da, q, s.clone().requires_grad_())),
    ]
    for match, call in bad:
        with pytest.raises(ValueError, match="^" + match):
            call()
    assert not launches


def test_host_tensors_are_refused():
    h = torch.zeros(3, 8)
    for call in (lambda: moe.swiglu(h), lambda: moe.swiglu_forward(h), lambda: moe.swiglu_backward(h, h, h)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
