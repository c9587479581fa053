"""Products of 8-bit integers with a few rows and very many columns (a
vocabulary's), where no rule for a small tile applies any more: up to 16 rows
are all of them rows behind the large tiles, of which there is none."""

from __future__ import annotations

import pytest
import torch

from gpu_helpers import log
from mixture_experts_expert_mm_amd import moe
from sort_reference import F64, HALF, U32

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes(seed, *shape):
    return torch.randint(-128, 128, shape, generator=gen(seed), dtype=torch.int8)


def scales(seed, *shape):
    return torch.rand(*shape, generator=gen(seed)) * 0.01 + 1e-4


def within(y, q, s, w, ws):
    """The sum becomes float32, two float32 products, one rounding."""
    want = (q.to(F64) @ w.to(F64).t()) * ws.to(F64) * s.to(F64)[:, None]
    over = (y.cpu().to(F64) - want).abs() - want.abs() * (3 * U32 + HALF[y.dtype]) * 1.01
    assert y.shape == want.shape and bool((over <= 0).all()), (float(over.max()), (over > 0).nonzero()[:4])


# 8 rows are streamed by a kernel of their own, 9 to 16 by that of the large tiles, 17 and more are a tile's; 512 tiles of
# 128 columns (two a CU) end at 65536
@pytest.mark.parametrize("M,N,K", [(8, 66000, 144), (9, 65536, 144), (9, 65540, 144), (9, 66000, 144), (16, 129281, 272), (16, 66003, 2064),
                                   (17, 70000, 128), (130, 66002, 144)])
@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
def test_product(M, N, K, y_dtype):
    log(f"[int8 wide] M={M} N={N} K={K} {y_dtype}")
    q, w, s, ws = codes(M, M, K), codes(N, N, K), scales(K, M), scales(K + 1, N)
    y = torch.full((M + 1, N), 7.0, dtype=TYPES[y_dtype], device="cuda")
    out = moe.int8_matmul(q.cuda(), s.cuda(), w.cuda(), ws.cuda(), y_dtype=y_dtype, y=y[:M])
    within(out, q, s, w, ws)
    assert bool((y[M] == 7.0).all())                     # (what lies behind the last row stays)


@pytest.mark.parametrize("M,N,K", [(9, 66000, 144), (16, 66001, 512), (16, 66000, 528)])
def test_linear(M, N, K):
    """From floating rows: quantised within the product up to 8192 values, before it beyond."""
    log(f"[int8 wide linear] M={M} N={N} K={K}")
    x, w, ws = torch.randn(M, K, generator=gen(M)).to(BF16).cuda(), codes(N, N, K).cuda(), scales(K + 1, N).cuda()
    q, s = moe.int8_quantize(x)
    y = moe.int8_linear(x, w, ws, y_dtype="f32")
    assert torch.equal(y, moe.int8_matmul(q, s, w, ws, y_dtype="f32"))
    within(y, q.cpu(), s.cpu(), w.cpu(), ws.cpu())


def test_groups():
    """Two groups of a few rows: tiles, none streamed."""
    M, N, K = 12, 66000, 144
    q, w, s, ws = codes(1, M, K), codes(2, 2, N, K), scales(3, M), scales(4, 2, N)
    off, cnt = torch.tensor([0, 5], dtype=torch.int32), torch.tensor([5, 7], dtype=torch.int32)
    y = moe.int8_matmul(q.cuda(), s.cuda(), w.cuda(), ws.cuda(), off.cuda(), cnt.cuda(), y_dtype="f32")
    within(y[:5], q[:5], s[:5], w[0], ws[0])
    within(y[5:], q[5:], s[5:], w[1], ws[1])
