"""The activation where its sigmoid leaves float32's normal numbers: accurate
down to 2^-126, and off by no more than that below."""

from __future__ import annotations

import pytest
import torch

import swiglu_reference as ref
from mixture_experts_expert_mm_amd import moe
from sort_reference import F64, HALF, U32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_gates_far_below_zero(dtype):
    g = torch.cat([-torch.arange(80.0, 92.0, 0.125), torch.tensor([-100.0, -1000.0, 80.0, 87.5, 89.0, 1000.0])]).to(dtype)
    u = 2.0 ** 14 if dtype == torch.float16 else 2.0 ** 100       # (large enough for every a to be a normal number)
    n = -(-g.numel() // 8) * 8
    h = torch.zeros(2, 2 * n, dtype=dtype)
    h[:, :g.numel()], h[0, n:], h[1, n:] = g, u, -u
    a = moe.swiglu(h.cuda()).cpu().to(F64)
    gate, up = h[:, :n].to(F64), h[:, n:].to(F64)
    want = gate * torch.sigmoid(gate) * up
    # the sigmoid's relative error and 2^-126 of its own, two products, one rounding
    err = want.abs() * (ref.SIG[dtype] + 4 * U32 + HALF[dtype]) * 1.01 + 2.0 ** -126 * gate.abs() * up.abs() * 1.01 + ref.TINY[dtype]
    # beyond the type's range (float16: 80 * 2^14 is above 65520) infinity is the rounded value
    out = want.to(dtype).isinf()
    assert torch.equal(a[out], want.to(dtype).to(F64)[out])
    diff, want, gate, err = (a - want)[~out].abs(), want[~out], gate[~out], err[~out]
    assert bool((diff <= err).all()), float((diff - err).max())
    fine = gate >= -87.3                                          # here the first part alone
    assert bool((diff <= want.abs() * (ref.SIG[dtype] + 4 * U32 + HALF[dtype]) * 1.01 + ref.TINY[dtype])[fine].all())
