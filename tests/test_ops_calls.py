"""How the operators' functions read their arguments, without a GPU: the checks, buffers and plans are the real
ones, the launches are recorded."""

from __future__ import annotations

import contextlib

import pytest
import torch

from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; the calls that would launch are listed as (name, arguments)."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    for name in ("mm_router", "mm_moe_few", "mm_block_quantize", "mm_block_gemm", "mm_block_linear"):
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def few_args(T=3, H=256, I=128, E=4, K=2):
    x = torch.zeros(T, H, dtype=BF16)
    w1, w2 = torch.zeros(E, 2 * I, H, dtype=BF16), torch.zeros(E, H, I, dtype=BF16)
    return (x, w1, w2), dict(topk_ids=torch.zeros(T, K, dtype=torch.int32), topk_weights=torch.zeros(T, K))


@pytest.mark.parametrize("y_dtype,want", [("bf16", BF16), ("f32", F32), ("fp32", F32), (B.MM_OUT_F32, F32),
                                          (B.MM_OUT_BF16, BF16)])
def test_y_has_the_type_that_the_plan_writes(launches, y_dtype, want):
    args, routes = few_args()
    y, _, _ = moe.moe_few(*args, y_dtype=y_dtype, **routes)
    plan, out = launches[-1][1][0], launches[-1][1][9]
    assert out is y and y.dtype == want
    assert plan.prob.y_dtype == (B.MM_OUT_F32 if want == F32 else B.MM_OUT_BF16)
    other = torch.zeros(3, 256, dtype=BF16 if want == F32 else F32)
    with pytest.raises(ValueError, match="y:"):
        moe.moe_few(*args, y_dtype=y_dtype, y=other, **routes)
    layer = moe.ExpertLayer(3, 256, 128, 4, 2, "bf16", y_dtype, device="cpu")
    assert layer.new_y().dtype == want
    layer.w1, layer.w2 = args[1:]
    assert layer.forward_few(args[0], **routes).dtype == want


@pytest.mark.parametrize("y_dtype", ["float32", "bfloat16", "", 2, -1])
def test_unknown_y_types_are_refused(launches, y_dtype):
    args, routes = few_args()
    with pytest.raises(B.MMError):
        moe.moe_few(*args, y_dtype=y_dtype, **routes)
    assert not launches


@pytest.mark.parametrize("name", ["x", "w1", "topk_weights"])
def test_tangents_are_refused(launches, name):
    """The tangent of forward mode would be dropped in silence, as a gradient would."""
    import torch.autograd.forward_ad as fw

    (x, w1, w2), routes = few_args()
    args = dict(x=x, w1=w1, w2=w2, **routes)
    with fw.dual_level():
        moe.moe_few(**args)                                  # none carries one
        n = len(launches)
        args[name] = fw.make_dual(args[name], torch.ones_like(args[name]))
        with pytest.raises(ValueError, match=f"{name}: .*tangent"):
            moe.moe_few(**args)
        assert len(launches) == n
        q = torch.zeros(2, 128, dtype=BF16)
        moe.block_quantize(q)
        with pytest.raises(ValueError, match="x: .*tangent"):
            moe.block_quantize(fw.make_dual(q, torch.ones_like(q)))


def test_counts_are_whole_numbers(launches):
    """A fraction of an expert is refused, not cut off."""
    (x, w1, w2), routes = few_args()
    wr = torch.zeros(4, 256, dtype=BF16)
    for kw in (dict(router_weight=wr, topk=2.5), dict(router_weight=wr, topk="2"), dict(routes, num_shared_experts=0.5)):
        with pytest.raises(ValueError, match="whole number"):
            moe.moe_few(x, w1, w2, **kw)
    with pytest.raises(ValueError, match="topk: .*whole number"):
        moe.route(x, wr, topk=1.5)
    assert not launches
    import numpy as np
    assert moe.route(x, wr, topk=np.int64(2))[0].shape == moe.route(x, wr, topk=2.0)[0].shape == (3, 2)
    assert moe.moe_few(x, w1, w2, router_weight=wr, topk=torch.tensor(2))[1].shape == (3, 2)


def overlapping(y_shape, x_shape, x_dtype, shift):
    """(y, x): two tensors of one buffer, x beginning `shift` bytes after y."""
    buf = torch.zeros(1 << 14, dtype=torch.uint8)
    n, m = 2 * y_shape[0] * y_shape[1], x_shape[0] * x_shape[1] * x_dtype.itemsize
    return buf[:n].view(BF16).view(y_shape), buf[shift:shift + m].view(x_dtype).view(x_shape)


@pytest.mark.parametrize("shift,ok", [(0, False), (512, False), (1008, False), (1024, True), (2048, True)])
def test_y_apart_from_the_inputs(launches, shift, ok):
    """Workgroups read the rows while others write y."""
    w, ws = torch.zeros(128, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 1)
    y, x = overlapping((4, 128), (4, 128), BF16, shift)
    assert moe.block_linear(x, w, ws, y=y) is y              # (reads x first where they overlap)
    y, q = overlapping((4, 128), (4, 128), torch.float8_e4m3fn, shift)
    if ok:
        assert moe.block_matmul(q, torch.zeros(4, 1), w, ws, y=y) is y
    else:
        with pytest.raises(ValueError, match="y: .*overlap"):
            moe.block_matmul(q, torch.zeros(4, 1), w, ws, y=y)
    (_, w1, w2), routes = few_args(T=2)
    y, gates = overlapping((2, 256), (2, 2), F32, shift)
    few = lambda x, y: moe.moe_few(x, w1, w2, y=y, topk_ids=routes["topk_ids"], topk_weights=gates)[0]
    if ok:
        assert few(torch.zeros(2, 256, dtype=BF16), y) is y
    else:
        with pytest.raises(ValueError, match="y: .*overlap"):
            few(torch.zeros(2, 256, dtype=BF16), y)


def test_the_layer_may_write_over_its_tokens(launches):
    """Linear1 has read x before Linear2 writes y; the weights stay apart."""
    (x, w1, w2), routes = few_args(T=2)
    assert moe.moe_few(x, w1, w2, y=x, **routes)[0] is x
    with pytest.raises(ValueError, match="y: .*overlap"):
        moe.moe_few(x, w1, w2, y=w2.view(-1, 256)[:2], **routes)
