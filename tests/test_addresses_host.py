"""Contiguous tensors that begin between two vectors (no GPU): every function
names the argument that it cannot take, before anything is launched."""

from __future__ import annotations

import contextlib

import pytest
import torch

import sort_reference as ref
from mixture_experts_expert_mm_amd import binding as B
from mixture_experts_expert_mm_amd import moe

BF16, F16, F32, I8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.int32
E4M3 = torch.float8_e4m3fn


@pytest.fixture
def launches(monkeypatch):
    """Host tensors pass as device ones; what would launch is listed by name."""
    seen = []
    monkeypatch.setattr(moe, "_rows", lambda name, x: (*x.shape, x.device))
    monkeypatch.setattr(moe, "_stream_of", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(moe, "_raw_stream", lambda device: 0)
    for name in B.EXPORTS:
        if hasattr(B, name) and not name.endswith(("_create", "_string", "_name")):
            monkeypatch.setattr(B, name, lambda *a, name=name, **kw: seen.append(name))
    return seen


def odd(t):
    """The same values at an address one element behind a multiple of 16 bytes."""
    buf = torch.empty(t.numel() + 32, dtype=t.dtype)
    at = (-(buf.data_ptr() // t.itemsize)) % 16 + 1
    o = buf[at:at + t.numel()].view(t.shape)
    o.copy_(t)
    assert o.is_contiguous() and o.data_ptr() % 16 == t.itemsize % 16
    return o


def arguments():
    T, H, I, E, K = 4, 256, 128, 3, 2
    ids = torch.zeros(T, K, dtype=I32)
    o = moe.TokenOrder(*ref.order(ids, E))
    x, rows, w, gates = torch.zeros(T, H, dtype=BF16), torch.zeros(T * K, H, dtype=BF16), torch.zeros(T, K), torch.zeros(T, K)
    h, da = torch.zeros(T, 2 * I, dtype=F16), torch.zeros(T, I, dtype=F16)
    q, qs, kept, ks = torch.zeros(T, H, dtype=I8), torch.zeros(T), torch.zeros(T, 2 * I, dtype=I8), torch.zeros(T, 2)
    w8, s8, y = torch.zeros(8, H, dtype=I8), torch.zeros(8), torch.zeros(T, 8, dtype=BF16)
    f8, fs, fw, fws, fy = (torch.zeros(T, H, dtype=E4M3), torch.zeros(T, 2), torch.zeros(128, H, dtype=E4M3), torch.zeros(1, 2),
                           torch.zeros(T, 128, dtype=BF16))
    w1, w2, wr = torch.zeros(E, 2 * I, H, dtype=BF16), torch.zeros(E, H, I, dtype=BF16), torch.zeros(E, H, dtype=BF16)
    e1, e2, s1, s2 = w1.to(E4M3), w2.to(E4M3), torch.zeros(E, 2 * I), torch.zeros(E, H)
    few = lambda **a: moe.moe_few(topk_ids=ids, topk_weights=w, **a)
    return [
        (lambda **a: moe.sort_tokens(topk_ids=ids, num_experts=E, **a), dict(x=x)),
        (lambda **a: moe.sort_rows(order=o, **a), dict(x=x)),
        (lambda **a: moe.combine_tokens(order=o, weights=gates, **a), dict(rows=rows)),
        (lambda **a: moe.combine_backward(order=o, weights=gates, **a), dict(dy=x, rows=rows)),
        (moe.swiglu, dict(h=h)), (moe.swiglu_forward, dict(h=h)),
        (lambda **a: moe.swiglu_backward(scales=ks, **a), dict(da=da, codes=kept)),
        (moe.int8_quantize, dict(x=x)),
        (lambda **a: moe.int8_matmul(s=qs, **a), dict(q=q, w=w8, ws=s8, y=y)),
        (moe.int8_linear, dict(x=x, w=w8, ws=s8, y=y)),
        (moe.block_quantize, dict(x=x)),
        (lambda **a: moe.block_matmul(s=fs, ws=fws, **a), dict(q=f8, w=fw, y=fy)),
        (lambda **a: moe.block_linear(ws=fws, **a), dict(x=x, w=fw, y=fy)),
        (lambda **a: moe.route(topk=2, **a), dict(x=x, weight=wr)),
        (few, dict(x=x, w1=w1, w2=w2, y=torch.zeros(T, H, dtype=BF16))),
        (few, dict(x=x, w1=e1, w2=e2, s1=s1, s2=s2)),
    ]


@pytest.mark.parametrize("i", range(16))
def test_an_argument_at_an_odd_address(launches, i):
    call, args = arguments()[i]
    call(**args)
    n = len(launches)
    assert n > 0
    for name in args:
        with pytest.raises(ValueError, match=f"^{name}: .*multiple of 16"):
            call(**{**args, name: odd(args[name])})
    assert len(launches) == n


def test_what_needs_no_such_address(launches):
    """Ids, weights, masks, scales of rows, and scales of channels that are read one by one."""
    T, H, E, K = 4, 256, 3, 2
    ids = torch.zeros(T, K, dtype=I32)
    o = moe.TokenOrder(*(odd(t) for t in ref.order(ids, E)))
    x, rows = torch.zeros(T, H), torch.zeros(T * K, H)
    moe.sort_tokens(x, odd(ids), E, active=odd(torch.ones(T, dtype=I8)))
    moe.sort_rows(x, o)
    moe.combine_tokens(rows, o, odd(torch.zeros(T, K)))
    moe.combine_backward(x, rows, o, odd(torch.zeros(T, K)))
    moe.swiglu_backward(torch.zeros(T, 128), torch.zeros(T, 256, dtype=I8), odd(torch.zeros(T, 2)))
    q = torch.zeros(T, H, dtype=I8)
    moe.int8_matmul(q, odd(torch.zeros(T)), torch.zeros(7, H, dtype=I8), odd(torch.zeros(7)))
    assert len(launches) == 6
