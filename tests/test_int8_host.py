"""Host side of the 8-bit integer product (no GPU): plans, refusals before any
HIP call, and how its functions read their arguments."""

from __future__ import annotations

import contextlib
import ctypes
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


@pytest.mark.parametrize("dims", [(0, 16, 16, 1), ((1 << 24) + 1, 16, 16, 1), (4, 0, 16, 1), (4, (1 << 20) + 1, 16, 1), (4, 16, 0, 1),
                                  (4, 16, 8, 1), (4, 16, 24, 1), (4, 16, 131072, 1), (4, 16, 16, 0), (4, 16, 16, 1025)])
def test_plan_refuses(dims):
    with pytest.raises(B.MMError) as ei:
        B.mm_int8_plan_create(*dims)
    assert ei.value.status == 1


def test_plan():
    assert ctypes.sizeof(B.MMInt8Problem) == 40 and ctypes.sizeof(B.MMInt8Plan) == 40 + 16 + 8 + 32
    p = B.mm_int8_plan_create(5, 1, 131056)
    assert p.workspace_bytes >= 5 * 131060 and p.dense_workspace_bytes == p.workspace_bytes
    p = B.mm_int8_plan_create(2, 64, 4096)                         # few rows: quantised inside the product, unless in groups
    assert p.workspace_bytes >= 2 * 4100 and p.dense_workspace_bytes == 0
    for kw in (dict(x_element=3), dict(y_element=3), dict(x_element=-1), dict(y_element=4)):
        with pytest.raises(B.MMError) as ei:
            B.mm_int8_plan_create(4, 16, 16, **kw)
        assert ei.value.status == 2


def test_entry_points_validate_before_any_hip_call(lib):
    P = ctypes.byref

    def call(fn, args, i, v):
        a = list(args)
        a[i] = v
        return fn(*a)

    args = [4, 32, 0, GOOD, GOOD, GOOD, None]
    for i, v in ((0, 0), (0, (1 << 24) + 1), (1, 0), (1, 8), (1, 24), (1, 131072), (3, None), (4, None), (5, None), (3, GOOD + 8),
                 (4, GOOD + 8), (5, GOOD + 2)):
        assert call(lib.mm_int8_quantize, args, i, v) == 1
    for v in (-1, 3):
        assert call(lib.mm_int8_quantize, args, 2, v) == 2
    p, gp = B.mm_int8_plan_create(40, 10, 32), B.mm_int8_plan_create(40, 10, 32, 3)
    bad = B.MMInt8Plan.from_buffer_copy(p)
    bad.prob.rows = 5
    args = [P(p), GOOD, GOOD, GOOD, GOOD, None, None, GOOD, None]
    for i in (1, 2, 3, 4, 7):
        assert call(lib.mm_int8_gemm, args, i, None) == 1
        assert call(lib.mm_int8_gemm, args, i, GOOD + 2) == 1
    for i in (5, 6):                                               # one group array without the other
        assert call(lib.mm_int8_gemm, args, i, GOOD) == 1
    for v in (P(bad), P(gp), None):                                # (several groups need their rows)
        assert call(lib.mm_int8_gemm, args, 0, v) == 1
    wide = B.mm_int8_plan_create(40, 12, 32)                       # scales of whole vectors are read as such
    assert call(lib.mm_int8_gemm, [P(wide)] + args[1:], 4, GOOD + 4) == 1
    args = [P(p), GOOD, GOOD, GOOD, None, None, GOOD, GOOD, 1 << 40, None]
    for i in (1, 2, 3, 6, 7):
        assert call(lib.mm_int8_linear, args, i, None) == 1
        assert call(lib.mm_int8_linear, args, i, GOOD + 2) == 1
    assert call(lib.mm_int8_linear, args, 4, GOOD) == 1 and call(lib.mm_int8_linear, args, 8, 16) == 3
    assert [B.mm_kernel_name(i) for i in (23, 24)] == ["int8_quantize", "int8_gemm"]


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; the calls that would launch are listed as (name, arguments)."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    for name in ("mm_int8_quantize", "mm_int8_gemm", "mm_int8_linear"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def test_what_is_launched(launches):
    x, w, ws = torch.zeros(5, 48, dtype=torch.float16), torch.zeros(7, 48, dtype=torch.int8), torch.zeros(7)
    q, s = moe.int8_quantize(x)
    assert q.shape == x.shape and q.dtype == torch.int8 and s.shape == (5,) and launches[-1][1][2] == B.MM_ELEMENT_F16
    for name, dt in (("bf16", torch.bfloat16), ("f16", torch.float16), ("f32", torch.float32)):
        y = moe.int8_matmul(q, s, w, ws, y_dtype=name)
        assert y.shape == (5, 7) and y.dtype == dt and launches[-1][1][0].prob.y_element == B.ELEMENT[dt]
    y = torch.zeros(5, 7, dtype=torch.bfloat16)
    assert moe.int8_linear(x, w, ws, y=y) is y
    assert launches[-1][1][0].prob.x_element == B.MM_ELEMENT_F16 and launches[-1][1][7] is None
    one = torch.zeros(1, dtype=torch.int32)
    for big, groups in ((torch.zeros(50, 48), ()), (x.float(), (one, one))):
        moe.int8_linear(big, w[None] if groups else w, ws[None] if groups else ws, *groups)
        plan = launches[-1][1][0]
        assert plan.prob.x_element == B.MM_ELEMENT_F32 and launches[-1][1][7].numel() == plan.workspace_bytes


def test_refusals(launches):
    x, w, ws = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    i32 = torch.zeros(3, dtype=torch.int32)
    w3, ws3 = torch.zeros(3, 8, 32, dtype=torch.int8), torch.zeros(3, 8)
    buf = torch.zeros(4096, dtype=torch.uint8)
    over = buf[:64].view(torch.bfloat16).view(4, 8)
    bad = [
        ("x", lambda: moe.int8_quantize(q)), ("x", lambda: moe.int8_quantize(x[:, :24].contiguous())), ("x", lambda: moe.int8_quantize(x[:, ::2])),
        ("x: .*gradient", lambda: moe.int8_quantize(x.clone().requires_grad_())),
        ("x: .*gradient", lambda: moe.int8_linear(x.clone().requires_grad_(), w, ws)),
        ("x", lambda: moe.int8_linear(x.double(), w, ws)), ("w", lambda: moe.int8_linear(x, w.float(), ws)),
        ("w", lambda: moe.int8_linear(x, w[:, :16], ws)), ("w", lambda: moe.int8_linear(x, None, ws)), ("ws", lambda: moe.int8_linear(x, w, ws[:5])),
        ("ws", lambda: moe.int8_linear(x, w, None)), ("ws", lambda: moe.int8_linear(x, w3, ws, i32, i32)),
        ("offsets, counts", lambda: moe.int8_linear(x, w3, ws3)), ("offsets, counts", lambda: moe.int8_linear(x, w, ws, i32)),
        ("offsets", lambda: moe.int8_linear(x, w3, ws3, i32[:2], i32)), ("counts", lambda: moe.int8_linear(x, w3, ws3, i32, i32.long())),
        ("q", lambda: moe.int8_matmul(x, s, w, ws)), ("s", lambda: moe.int8_matmul(q, s[:3], w, ws)), ("s", lambda: moe.int8_matmul(q, s[:, None], w, ws)),
        ("y_dtype", lambda: moe.int8_matmul(q, s, w, ws, y_dtype="fp64")), ("y_dtype", lambda: moe.int8_matmul(q, s, w, ws, y_dtype=1)),
        ("y", lambda: moe.int8_matmul(q, s, w, ws, y=torch.zeros(4, 8))), ("y", lambda: moe.int8_matmul(q, s, w, ws, y=torch.zeros(4, 9, dtype=torch.bfloat16))),
        ("y: overlaps", lambda: moe.int8_linear(buf[32:288].view(torch.bfloat16).view(4, 32), w, ws, y=over)),
        ("y: overlaps", lambda: moe.int8_matmul(buf[:128].view(torch.int8).view(4, 32), s, w, ws, y=over)),
    ]
    for match, call in bad:
        with pytest.raises(ValueError, match="^" + match):
            call()
    for K in (0, 8, 131072):
        with pytest.raises(B.MMError):
            moe.int8_matmul(torch.zeros(4, K, dtype=torch.int8), s, torch.zeros(8, K, dtype=torch.int8), ws)
    assert not launches


def test_host_tensors_are_refused():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    for call in (lambda: moe.int8_quantize(x), lambda: moe.int8_linear(x, None, None), lambda: moe.int8_matmul(x, None, None, None)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
