"""Outputs over inputs: the calls that allow it give what they give apart."""

from __future__ import annotations

import pytest
import torch

from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("M,N,K", [(1, 1 << 17, 1024), (1, 8192, 8192), (8, 1024, 1024), (3, 40000, 2048), (600, 2048, 2048)])
@pytest.mark.parametrize("at", ["front", "middle"])
def test_linear_over_its_rows(M, N, K, at):
    """x inside y's memory, with more workgroups than run at once."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.float8_e4m3fn)
    ws = torch.rand(-(-N // 128), K // 128, generator=g, device="cuda") * 0.01
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    want = moe.block_linear(x, w, ws)
    y = torch.zeros(M, N, dtype=BF16, device="cuda")
    first = 0 if at == "front" else (M * N - M * K) // 2 // 64 * 64
    inside = y.view(-1)[first:first + M * K].view(M, K)
    for _ in range(3):
        y.zero_()
        inside.copy_(x)
        assert moe.block_linear(inside, w, ws, y=y) is y
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T,y_dtype", [(1, "bf16"), (16, "bf16"), (40, "bf16")])
def test_layer_over_its_tokens(T, y_dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    E, H, I, K = 8, 1024, 512, 2
    w1 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5).to(BF16)
    wr = (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    want, ids, wts = moe.moe_few(x, w1, w2, router_weight=wr, topk=K)
    for routes in (dict(router_weight=wr, topk=K), dict(topk_ids=ids, topk_weights=wts)):
        y = x.clone()
        assert moe.moe_few(y, w1, w2, y=y, **routes)[0] is y
        assert torch.equal(y, want)
