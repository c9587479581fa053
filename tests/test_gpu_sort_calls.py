"""Sorted tokens: calls on the GPU that their other tests leave out."""

from __future__ import annotations

import pytest
import torch

import sort_reference as ref
from mixture_experts_expert_mm_amd import moe

pytestmark = pytest.mark.gpu

F16, F64 = torch.float16, torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_recorded_calls_under_capture():
    """Every argument is as it has to be: what is refused is the capture."""
    ids = torch.randint(0, 3, (6, 2), generator=gen(1), dtype=torch.int32).cuda()
    x = torch.randn(6, 16, device="cuda", requires_grad=True)
    rows, order = moe.sort_tokens(x.detach(), ids, 3)
    w = torch.rand(6, 2, device="cuda", requires_grad=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (lambda: moe.sort_tokens(x, ids, 3), lambda: moe.sort_rows(x, order), lambda: moe.combine_tokens(rows, order, w),
                     lambda: moe.swiglu(x)):
            with pytest.raises(RuntimeError, match="capture"):
                call()
        with torch.no_grad():
            again, o = moe.sort_tokens(x, ids, 3)
            y = moe.combine_tokens(again, o, w)
    for _ in range(3):
        graph.replay()
        want = moe.combine_tokens(rows, order, w).detach()
        torch.cuda.synchronize()
        assert torch.equal(again, rows) and torch.equal(y, want)


@pytest.mark.parametrize("T", [5, 9000])
@pytest.mark.parametrize("weighted", [False, True])
def test_tokens_that_name_one_expert_every_time(T, weighted):
    """An id that a token names several times is as many routes, each with a weight of its own."""
    E, K = 6, 3
    ids = torch.full((T, K), E - 1, dtype=torch.int32)
    x, w = torch.randn(T, 40, generator=gen(T)).to(F16), torch.rand(T, K, generator=gen(T + 1))
    rows, order = moe.sort_tokens(x.cuda(), ids.cuda(), E)
    y = moe.combine_tokens(rows, order, w.cuda() if weighted else None)
    want, err = ref.combine(rows.cpu(), ref.order(ids, E)[2], w if weighted else None)
    assert bool(((y.cpu().to(F64) - want).abs() <= err).all())
